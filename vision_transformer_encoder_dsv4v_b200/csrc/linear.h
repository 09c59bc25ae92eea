// Interface between the Linear layer's entry points (linear.cu) and its tcgen05 GEMM (linear_tc.cu).
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <stdint.h>

#include "dsv4v.h"

namespace dsv4v {

// What happens to an accumulator element: v + bias[col], kept in z, activated, residual added,
// rounded once into y.
struct LinearEpilogue {
  __nv_bfloat16* y;
  int64_t ld_y;
  const float* bias;               // 16-byte aligned, or NULL
  const __nv_bfloat16* residual;   // or NULL; may be y itself
  int64_t ld_residual;
  __nv_bfloat16* z;                // or NULL
  int64_t ld_z;
  int act;
  bool vec_io;                     // the rows of y, residual and z are 16-byte aligned
};

// out[f] = the sum over strips of sums[strip][f], f < M; out NULL: none.
struct ColumnSums {
  const float* sums = nullptr;
  int strips = 0;
  float* out = nullptr;
};

enum LinearForm {
  LINEAR_FORWARD,      // D[rows, out] = x . W^T: both operands K-major
  LINEAR_FORWARD_SWAPPED,  // D[out, rows] = W . x^T, of up to 32 rows, stored as y
  LINEAR_INPUT_GRAD,   // dx[rows, in] = dz . W: dz K-major, W MN-major
  LINEAR_WEIGHT_GRAD,  // dW[out, in] = dz^T . x: both MN-major
  LINEAR_BOTH_GRADS,   // dx and dW in one launch
};

// How a launch is cut up; the second entries are dW's of LINEAR_BOTH_GRADS.
struct LinearPlan {
  int pair = 0, bn = 0, ks = 1;  // CTA pairs; columns of a tile; K splits (cluster size)
  int swap = 0;                  // the forward as LINEAR_FORWARD_SWAPPED: its M are the features
  int tiles_m[2] = {}, tiles_n[2] = {}, kb_total[2] = {} /* stages */, grid = 0;
  int units = 0;                 // of LINEAR_BOTH_GRADS: CTAs (pairs) of dx
  int a_rows = 0;                // rows of the boxes of a K-major A
  double us = 0;                 // estimated time
};
struct LinearMaps {
  CUtensorMap a[2], b[2];
};
struct LinearProduct {
  int M, N;
  LinearEpilogue e;
};

// Tile, pairing and split of D[M, N] over a contraction of K, on `sms` SMs.
LinearPlan plan_linear(LinearForm form, int64_t M, int64_t N, int64_t K, int sms);
// The same for both gradients of a layer in one launch.
LinearPlan plan_linear_both(int64_t rows, int64_t in, int64_t out, int sms);
// Depth of a stage, and rows of the boxes of A's and B's tensor maps (for an MN-major operand, rows
// of the contraction) under a plan.
inline int linear_depth(const LinearPlan& p) { return p.bn <= 192 ? 128 : 64; }
inline int linear_box_a(const LinearPlan& p, bool a_mn) { return a_mn ? linear_depth(p) : p.a_rows; }
inline int linear_box_b(const LinearPlan& p, bool b_mn) { return b_mn ? linear_depth(p) : (p.pair ? p.bn / 2 : p.bn); }

// The forward of a few rows without tensor cores, and whether it is taken.
bool linear_is_few(int64_t M, int64_t N, int64_t K, int sms);
cudaError_t launch_linear_few(const void* x, int64_t ld_x, const void* w, int64_t ld_w, int M, int N, int K, const LinearEpilogue& e,
                              int sms, cudaStream_t s);

cudaError_t launch_linear(LinearForm form, const LinearPlan& plan, const LinearMaps& maps, const LinearProduct* products,
                          const ColumnSums& cs, uint32_t* err, cudaStream_t s);

// The same for fp32 matrices (linear_f32.cu).
struct EpilogueF32 {
  float* y;
  int64_t ld_y;
  const float* bias;
  const float* residual;
  int64_t ld_residual;
  float* z;
  int64_t ld_z;
  int act;
};
// D[M, N] over a contraction of K.  a is stored [M, K], for the weight gradient [K, M]; b [N, K], for the
// gradients [K, N].
struct ProductF32 {
  const float* a;
  int64_t lda;
  const float* b;
  int64_t ldb;
  int64_t M, N, K;
  EpilogueF32 e;
};
cudaError_t launch_linear_f32(LinearForm form, const ProductF32& p, const ColumnSums& cs, uint32_t* err, int sms, cudaStream_t s);
// Both gradients: in one launch where their tiles fit the SMs together, else one after the other.
cudaError_t launch_linear_f32_grads(const ProductF32& dx, const ProductF32& dw, const ColumnSums& cs, uint32_t* err, int sms,
                                    cudaStream_t s);

}  // namespace dsv4v
