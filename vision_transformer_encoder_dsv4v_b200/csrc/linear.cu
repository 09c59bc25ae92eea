// Entry points of the Linear layer (forward and backward) and the kernels around its products: the
// gradient of the activation, with the bias gradient's sums.
#include <algorithm>
#include <type_traits>

#include "common.cuh"
#include "internal.h"
#include "linear.h"

// No pointer here is __restrict__: the kernels start before their predecessor ends, and a load that
// the compiler may take for invariant could move ahead of the wait for it.
namespace dsv4v {

namespace {

// ---------------------------------------------------------------------------- activation gradient
// dz = dy act'(z).  The bf16 path takes its exponentials and reciprocals from the MUFU pipe (a few
// 2^-23, against the 2^-9 of the bf16 result); the fp32 path calls erff and expf.
template <int ACT, bool EXACT>
__device__ __forceinline__ float derivative(float z) {
  if constexpr (ACT == DSV4V_ACT_GELU) {
    // Phi(z) + z phi(z)
    if constexpr (EXACT)
      return 0.5f * (1.0f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
    // erfc by Abramowitz and Stegun 7.1.26, |error| <= 1.5e-7; its e^(-z^2 / 2) serves phi too
    const float t = rcp_approx(fmaf(0.3275911f * 0.70710678118654752f, fabsf(z), 1.0f));
    float q = fmaf(1.061405429f, t, -1.453152027f);
    q = fmaf(q, t, 1.421413741f);
    q = fmaf(q, t, -0.284496736f);
    q = fmaf(q, t, 0.254829592f);
    const float ex = ex2_approx(z * z * -0.72134752044448170f);
    const float tail = 0.5f * q * t * ex;
    return fmaf(z * 0.39894228040143268f, ex, z >= 0.0f ? 1.0f - tail : tail);
  }
  if constexpr (ACT == DSV4V_ACT_SILU) {
    // s (1 + z (1 - s)), s the logistic of z; far below zero s vanishes before z (1 - s) grows
    const float s = EXACT ? 1.0f / (1.0f + expf(-z)) : rcp_approx(1.0f + ex2_approx(z * -1.4426950408889634f));
    return s * fmaf(z, 1.0f - s, 1.0f);
  }
  return 1.0f;
}

// Eight elements of a row: 16-byte pieces as they are loaded, and their values.
template <class T>
struct Eight;
template <>
struct Eight<__nv_bfloat16> {
  uint4 q;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { q = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
    v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
  }
};
template <>
struct Eight<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void values(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
};
__device__ __forceinline__ float value_of(__nv_bfloat16 x) { return __bfloat162float(x); }
__device__ __forceinline__ float value_of(float x) { return x; }
// dz lies in the workspace, its rows padded to 8 elements: whole pieces always fit.
__device__ __forceinline__ void put8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void put8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

constexpr int kDzCols = 256;  // columns of a CTA: 32 threads of 8, by 8 rows at a time

// One pass over dy (and z): writes dz where it is wanted and, per strip of rows, the column sums of
// the unrounded dz, whose strips k_column_sums adds in order.  In bf16, dz is rounded because it is an operand
// of tcgen05 products beside the bf16 w and x: dx and dw are then two roundings from exact (2.35e-3 of their
// norm) instead of one (1.66e-3).  As two bf16 parts it would cost both products twice (of the 495 us of 8192 x
// 4608 -> 4096 they are about 460).  HBM bounds it (8192 x 4096 bf16, dy and z
// read: 25 us, 5.3 TB/s, with four CTAs an SM of two rows in flight a thread; 34 us with two CTAs of
// four).  VEC: rows are 16-byte aligned.
template <class T, int ACT, bool VEC>
__global__ void __launch_bounds__(256, VEC ? (sizeof(T) == 2 ? 4 : 2) : 1)
    k_linear_dz(const T* dy, int64_t ld_dy, const T* z, int64_t ld_z, T* dz, int64_t ld_dz, float* sums, int64_t rows, int n,
                int64_t strip) {
  launch_dependents();
  grid_dependency_wait();
  __shared__ float s[8][kDzCols + 8];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int col = blockIdx.x * kDzCols + cx * 8;
  const int cnt = min(8, n - col);
  float acc[8] = {0, 0, 0, 0, 0, 0, 0, 0};
  if (cnt > 0) {
    const int64_t r0 = static_cast<int64_t>(blockIdx.y) * strip, r1 = min(rows, r0 + strip);
    auto finish = [&](int64_t r, float (&g)[8], const float (&v)[8]) {
      if constexpr (ACT != DSV4V_ACT_NONE) {
#pragma unroll
        for (int j = 0; j < 8; ++j) g[j] *= derivative<ACT, sizeof(T) == 4>(v[j]);
      }
      if (dz) put8(dz + r * ld_dz + col, g);
#pragma unroll
      for (int j = 0; j < 8; ++j) acc[j] += g[j];
    };
    int64_t r = r0 + ry;
    if (VEC && cnt == 8) {
      constexpr int U = sizeof(T) == 2 ? 2 : 4;  // rows in flight
      auto batch = [&](auto count) {
        constexpr int C = decltype(count)::value;
        Eight<T> qg[C], qv[C];
#pragma unroll
        for (int u = 0; u < C; ++u) {
          qg[u].load(dy + (r + 8 * u) * ld_dy + col);
          if constexpr (ACT != DSV4V_ACT_NONE) qv[u].load(z + (r + 8 * u) * ld_z + col);
        }
#pragma unroll
        for (int u = 0; u < C; ++u) {
          float g[8], v[8] = {};
          qg[u].values(g);
          if constexpr (ACT != DSV4V_ACT_NONE) qv[u].values(v);
          finish(r + 8 * u, g, v);
        }
      };
      for (; r + 8 * (U - 1) < r1; r += 8 * U) batch(std::integral_constant<int, U>());
      for (; r < r1; r += 8) batch(std::integral_constant<int, 1>());
    }
    for (; r < r1; r += 8) {
      float g[8], v[8] = {};
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int at = col + min(j, cnt - 1);
        g[j] = value_of(dy[r * ld_dy + at]);
        if constexpr (ACT != DSV4V_ACT_NONE) v[j] = value_of(z[r * ld_z + at]);
        if (j >= cnt) g[j] = 0.0f;
      }
      finish(r, g, v);
    }
  }
  if (!sums) return;
#pragma unroll
  for (int j = 0; j < 8; ++j) s[ry][cx * 8 + j] = acc[j];
  __syncthreads();
  const int c = blockIdx.x * kDzCols + threadIdx.x;
  if (c >= n) return;
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) t += s[i][threadIdx.x];
  sums[static_cast<int64_t>(blockIdx.y) * n + c] = t;
}

__global__ void __launch_bounds__(256) k_column_sums(const float* sums, int strips, int n, float* out) {
  launch_dependents();
  grid_dependency_wait();
  __shared__ float s[8][33];
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float t = 0.0f;
  if (c < n)
#pragma unroll 4
    for (int i = ry; i < strips; i += 8) t += sums[static_cast<int64_t>(i) * n + c];
  s[ry][cx] = t;
  __syncthreads();
  if (ry != 0 || c >= n) return;
  t = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) t += s[i][cx];
  out[c] = t;
}

// ---------------------------------------------------------------------------- host side
bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
size_t up256(size_t x) { return (x + 255) & ~size_t(255); }

constexpr int64_t kMaxRows = int64_t(1) << 30;
constexpr int kMaxWidth = 1 << 20;  // 64-column tiles along a grid's y dimension stay in range

struct Layer {
  int64_t rows, k, n, ld_x, ld_w, ld_residual, ld_z, ld_y;
  int act;
  bool bf16;
  size_t es;
};

dsv4v_status check_layer(const dsv4v_linear* l, Layer& o) {
  if (!l || l->rows < 0 || l->rows > kMaxRows || l->in_features < 1 || l->out_features < 1) return DSV4V_ERR_INVALID_ARG;
  if (l->activation != DSV4V_ACT_NONE && l->activation != DSV4V_ACT_GELU && l->activation != DSV4V_ACT_SILU)
    return DSV4V_ERR_INVALID_ARG;
  if (l->dtype != DSV4V_F32 && l->dtype != DSV4V_BF16) return DSV4V_ERR_INVALID_ARG;
  if (l->in_features > kMaxWidth || l->out_features > kMaxWidth) return DSV4V_ERR_UNSUPPORTED;
  o.rows = l->rows;
  o.k = l->in_features;
  o.n = l->out_features;
  o.act = l->activation;
  o.bf16 = l->dtype == DSV4V_BF16;
  o.es = o.bf16 ? 2 : 4;
  const int64_t given[5] = {l->ld_x, l->ld_w, l->ld_residual, l->ld_z, l->ld_y}, least[5] = {o.k, o.k, o.n, o.n, o.n};
  int64_t* lds[5] = {&o.ld_x, &o.ld_w, &o.ld_residual, &o.ld_z, &o.ld_y};
  for (int i = 0; i < 5; ++i) {
    *lds[i] = given[i] == 0 ? least[i] : given[i];
    if (*lds[i] < least[i]) return DSV4V_ERR_INVALID_ARG;
    if (*lds[i] > (int64_t(1) << 32)) return DSV4V_ERR_UNSUPPORTED;
  }
  // TMA takes the rows of x, W (and of dx, dW's operands) in 16-byte steps.
  if (o.bf16 && (o.ld_x % 8 || o.ld_w % 8)) return DSV4V_ERR_UNSUPPORTED;
  return DSV4V_OK;
}

int64_t dz_ld(const Layer& l) { return (l.n + 7) / 8 * 8; }

// Strips of rows of the dz pass: about four CTAs an SM, at least 16 rows each.
int dz_strips(const Layer& l, int sms) {
  const int64_t across = (l.n + kDzCols - 1) / kDzCols;
  return static_cast<int>(std::max<int64_t>(1, std::min<int64_t>((l.rows + 15) / 16, 4ll * sms / across)));
}

struct BackwardLayout {
  size_t dz, sums, total;
};
BackwardLayout backward_layout(const Layer& l, int sms) {
  BackwardLayout b{};
  b.sums = up256(static_cast<size_t>(l.rows) * dz_ld(l) * l.es);
  b.total = b.sums + up256(static_cast<size_t>(dz_strips(l, sms)) * l.n * sizeof(float));
  return b;
}

dsv4v_status cuda_status(cudaError_t e) { return e == cudaSuccess ? DSV4V_OK : DSV4V_ERR_CUDA; }

// A bf16 operand and its row stride.
struct Operand {
  const void* p;
  int64_t ld;
};

// The tensor maps of D[M, N] over a contraction of K.  a is stored [M, K] or, MN-major, [K, M]; b [N, K]
// or [K, N].
bool operand_maps(const LinearPlan& plan, bool a_mn, bool b_mn, Operand a, Operand b, int64_t M, int64_t N, int64_t K, CUtensorMap* ta,
                  CUtensorMap* tb) {
  const int box_a = linear_box_a(plan, a_mn), box_b = linear_box_b(plan, b_mn);
  return tensor_map_bf16(a.p, a_mn ? K : M, a_mn ? M : K, box_a, a.ld, ta) && tensor_map_bf16(b.p, b_mn ? K : N, b_mn ? N : K, box_b, b.ld, tb);
}

// One bf16 product of the layer.
dsv4v_status gemm(LinearForm form, Operand a, Operand b, int64_t M, int64_t N, int64_t K, const LinearEpilogue& e, cudaStream_t s,
                  const ColumnSums& cs = ColumnSums()) {
  int sms = 0;
  uint32_t* err = nullptr;
  if (!query_device(&sms, &err)) return DSV4V_ERR_CUDA;
  const LinearPlan plan = plan_linear(form, M, N, K, sms);
  if (plan.bn == 0) return DSV4V_ERR_UNSUPPORTED;
  if (plan.swap) {
    form = LINEAR_FORWARD_SWAPPED;
    std::swap(a, b);
    std::swap(M, N);
  }
  LinearMaps maps;
  if (!operand_maps(plan, form == LINEAR_WEIGHT_GRAD, form == LINEAR_INPUT_GRAD || form == LINEAR_WEIGHT_GRAD, a, b, M, N, K, &maps.a[0], &maps.b[0])) return DSV4V_ERR_CUDA;
  const LinearProduct product{static_cast<int>(M), static_cast<int>(N), e};
  return cuda_status(launch_linear(form, plan, maps, &product, cs, err, s));
}

// Both bf16 gradients: in one launch where that is estimated to be sooner done, as for small layers,
// whose tiles leave SMs idle in each of two launches (784 rows, 1024 -> 2816: 19.3 us one after the
// other, 13.5 us together), else one after the other.
dsv4v_status gemm_grads(const Layer& l, Operand dz, const void* x, const void* w, const LinearEpilogue& dx, const LinearEpilogue& dw,
                        const ColumnSums& cs, cudaStream_t s) {
  int sms = 0;
  uint32_t* err = nullptr;
  if (!query_device(&sms, &err)) return DSV4V_ERR_CUDA;
  const LinearPlan px = plan_linear(LINEAR_INPUT_GRAD, l.rows, l.k, l.n, sms), pw = plan_linear(LINEAR_WEIGHT_GRAD, l.n, l.k, l.rows, sms);
  const LinearPlan both = plan_linear_both(l.rows, l.k, l.n, sms);
  if (px.bn == 0 || pw.bn == 0) return DSV4V_ERR_UNSUPPORTED;
  const LinearProduct products[2] = {{static_cast<int>(l.rows), static_cast<int>(l.k), dx}, {static_cast<int>(l.n), static_cast<int>(l.k), dw}};
  const bool one = both.bn && both.us < px.us + pw.us;
  LinearMaps maps;
  const LinearPlan& p0 = one ? both : px;
  const LinearPlan& p1 = one ? both : pw;
  if (!operand_maps(p0, false, true, dz, Operand{w, l.ld_w}, l.rows, l.k, l.n, &maps.a[0], &maps.b[0]) ||
      !operand_maps(p1, true, true, dz, Operand{x, l.ld_x}, l.n, l.k, l.rows, &maps.a[1], &maps.b[1]))
    return DSV4V_ERR_CUDA;
  if (one) return cuda_status(launch_linear(LINEAR_BOTH_GRADS, both, maps, products, cs, err, s));
  if (launch_linear(LINEAR_INPUT_GRAD, px, maps, products, ColumnSums(), err, s) != cudaSuccess) return DSV4V_ERR_CUDA;
  maps.a[0] = maps.a[1];
  maps.b[0] = maps.b[1];
  return cuda_status(launch_linear(LINEAR_WEIGHT_GRAD, pw, maps, products + 1, cs, err, s));
}

dsv4v_status gemm_f32(LinearForm form, const ProductF32& p, cudaStream_t s, const ColumnSums& cs = ColumnSums()) {
  int sms = 0;
  uint32_t* err = nullptr;
  if (!query_device(&sms, &err)) return DSV4V_ERR_CUDA;
  return cuda_status(launch_linear_f32(form, p, cs, err, sms, s));
}

bool rows16(const void* p, int64_t ld) { return !p || (aligned_to(p, 16) && ld % 8 == 0); }

dsv4v_status forward(const Layer& l, const void* x, const void* w, const float* bias, const void* residual, void* z, void* y,
                     cudaStream_t s) {
  if (!l.bf16) {
    const EpilogueF32 e{static_cast<float*>(y), l.ld_y, bias, static_cast<const float*>(residual), l.ld_residual,
                        static_cast<float*>(z), l.ld_z, l.act};
    return gemm_f32(LINEAR_FORWARD, ProductF32{static_cast<const float*>(x), l.ld_x, static_cast<const float*>(w), l.ld_w, l.rows, l.n, l.k, e}, s);
  }
  LinearEpilogue e{};
  e.y = static_cast<__nv_bfloat16*>(y);
  e.ld_y = l.ld_y;
  e.bias = bias;
  e.residual = static_cast<const __nv_bfloat16*>(residual);
  e.ld_residual = l.ld_residual;
  e.z = static_cast<__nv_bfloat16*>(z);
  e.ld_z = l.ld_z;
  e.act = l.act;
  int sms = 0;
  if (!query_device(&sms, nullptr)) return DSV4V_ERR_CUDA;
  if (linear_is_few(l.rows, l.n, l.k, sms))
    return cuda_status(launch_linear_few(x, l.ld_x, w, l.ld_w, static_cast<int>(l.rows), static_cast<int>(l.n), static_cast<int>(l.k), e,
                                         sms, s));
  e.vec_io = rows16(y, l.ld_y) && rows16(residual, l.ld_residual) && rows16(z, l.ld_z);
  return gemm(LINEAR_FORWARD, Operand{x, l.ld_x}, Operand{w, l.ld_w}, l.rows, l.n, l.k, e, s);
}

template <class T, int ACT, bool VEC>
cudaError_t launch_dz_vec(const Layer& l, const void* d_y, const void* z, void* dz, float* sums, int strips, cudaStream_t s) {
  const int64_t strip = (l.rows + strips - 1) / strips;
  return launch_pdl(k_linear_dz<T, ACT, VEC>, dim3(static_cast<unsigned>((l.n + kDzCols - 1) / kDzCols), static_cast<unsigned>(strips)),
                    dim3(256), 0, s, static_cast<const T*>(d_y), l.ld_y, static_cast<const T*>(z), l.ld_z, static_cast<T*>(dz),
                    dz_ld(l), sums, l.rows, static_cast<int>(l.n), strip);
}

template <class T, int ACT>
cudaError_t launch_dz_act(const Layer& l, const void* d_y, const void* z, void* dz, float* sums, int strips, cudaStream_t s) {
  const bool vec = aligned_to(d_y, 16) && l.ld_y * sizeof(T) % 16 == 0 &&
                   (ACT == DSV4V_ACT_NONE || (aligned_to(z, 16) && l.ld_z * sizeof(T) % 16 == 0));
  return vec ? launch_dz_vec<T, ACT, true>(l, d_y, z, dz, sums, strips, s) : launch_dz_vec<T, ACT, false>(l, d_y, z, dz, sums, strips, s);
}

template <class T>
cudaError_t launch_dz(const Layer& l, const void* d_y, const void* z, void* dz, float* sums, int strips, cudaStream_t s) {
  if (l.act == DSV4V_ACT_GELU) return launch_dz_act<T, DSV4V_ACT_GELU>(l, d_y, z, dz, sums, strips, s);
  if (l.act == DSV4V_ACT_SILU) return launch_dz_act<T, DSV4V_ACT_SILU>(l, d_y, z, dz, sums, strips, s);
  return launch_dz_act<T, DSV4V_ACT_NONE>(l, d_y, z, dz, sums, strips, s);
}

dsv4v_status backward(const Layer& l, const void* x, const void* w, const void* z, const void* d_y, void* dx, void* dw, float* db,
                      uint8_t* ws, const BackwardLayout& bl, int sms, cudaStream_t s) {
  if (l.rows == 0) {  // sums over no rows
    if (dw && cudaMemset2DAsync(dw, l.ld_w * l.es, 0, l.k * l.es, l.n, s) != cudaSuccess) return DSV4V_ERR_CUDA;
    if (db && cudaMemsetAsync(db, 0, l.n * sizeof(float), s) != cudaSuccess) return DSV4V_ERR_CUDA;
    return DSV4V_OK;
  }
  // dz is d_y itself without an activation, where TMA can take its rows.
  const bool products = dx || dw;
  const bool own_dz = l.act != DSV4V_ACT_NONE || (l.bf16 && !rows16(d_y, l.ld_y));
  const bool write_dz = products && own_dz;
  const int strips = dz_strips(l, sms);
  const bool sums_in_gemm = dw && db;  // the weight gradient's kernel adds the strips up
  if (write_dz || db) {
    float* sums = db ? reinterpret_cast<float*>(ws + bl.sums) : nullptr;
    void* dz = write_dz ? ws + bl.dz : nullptr;
    const cudaError_t e = l.bf16 ? launch_dz<__nv_bfloat16>(l, d_y, z, dz, sums, strips, s) : launch_dz<float>(l, d_y, z, dz, sums, strips, s);
    if (e != cudaSuccess) return DSV4V_ERR_CUDA;
    if (db && !sums_in_gemm && launch_pdl(k_column_sums, dim3(static_cast<unsigned>((l.n + 31) / 32)), dim3(256), 0, s, static_cast<const float*>(sums),
                         strips, static_cast<int>(l.n), db) != cudaSuccess)
      return DSV4V_ERR_CUDA;
  }
  ColumnSums cs;
  if (sums_in_gemm) cs = ColumnSums{reinterpret_cast<const float*>(ws + bl.sums), strips, db};
  const void* dz = write_dz ? static_cast<const void*>(ws + bl.dz) : d_y;
  const int64_t ld_dz = write_dz ? dz_ld(l) : l.ld_y;
  if (!l.bf16) {
    const float* z32 = static_cast<const float*>(dz);
    ProductF32 px{z32, ld_dz, static_cast<const float*>(w), l.ld_w, l.rows, l.k, l.n, {}};
    ProductF32 pw{z32, ld_dz, static_cast<const float*>(x), l.ld_x, l.n, l.k, l.rows, {}};
    px.e.y = static_cast<float*>(dx);
    px.e.ld_y = l.ld_x;
    pw.e.y = static_cast<float*>(dw);
    pw.e.ld_y = l.ld_w;
    if (dx && dw) {
      uint32_t* err = nullptr;
      if (!query_device(nullptr, &err)) return DSV4V_ERR_CUDA;
      return cuda_status(launch_linear_f32_grads(px, pw, cs, err, sms, s));
    }
    if (dx) return gemm_f32(LINEAR_INPUT_GRAD, px, s);
    return dw ? gemm_f32(LINEAR_WEIGHT_GRAD, pw, s, cs) : DSV4V_OK;
  }
  LinearEpilogue ex{}, ew{};
  ex.y = static_cast<__nv_bfloat16*>(dx);
  ex.ld_y = l.ld_x;
  ex.vec_io = rows16(dx, l.ld_x);
  ew.y = static_cast<__nv_bfloat16*>(dw);
  ew.ld_y = l.ld_w;
  ew.vec_io = rows16(dw, l.ld_w);
  const Operand z_op{dz, ld_dz};
  if (dx && dw) return gemm_grads(l, z_op, x, w, ex, ew, cs, s);
  if (dx) return gemm(LINEAR_INPUT_GRAD, z_op, Operand{w, l.ld_w}, l.rows, l.k, l.n, ex, s);
  if (dw) return gemm(LINEAR_WEIGHT_GRAD, z_op, Operand{x, l.ld_x}, l.n, l.k, l.rows, ew, s, cs);
  return DSV4V_OK;
}

// Runs `f`, turning an exception (the descriptor cache's allocation) into a status: none may leave
// a C entry.
template <class F>
dsv4v_status guarded(F&& f) {
  try {
    return f();
  } catch (...) {
    return DSV4V_ERR_CUDA;
  }
}

}  // namespace

}  // namespace dsv4v

using namespace dsv4v;

extern "C" {

dsv4v_status dsv4v_linear_forward(const dsv4v_linear* layer, const void* x, const void* w, const float* bias, const void* residual,
                                  void* z, void* y, void* stream) {
  Layer l;
  const dsv4v_status st = check_layer(layer, l);
  if (st != DSV4V_OK) return st;
  if (l.rows == 0) return DSV4V_OK;
  const size_t in = l.bf16 ? 16 : 4;
  if (!x || !w || !y || !aligned_to(x, in) || !aligned_to(w, in) || !aligned_to(y, l.es) || (bias && !aligned_to(bias, 16)) ||
      (residual && !aligned_to(residual, l.es)) || (z && !aligned_to(z, l.es)))
    return DSV4V_ERR_INVALID_ARG;
  if (y == x || y == w || z == x || z == w || z == y || (z && z == residual) || (residual == y && l.ld_residual != l.ld_y)) return DSV4V_ERR_INVALID_ARG;
  return guarded([&] { return forward(l, x, w, bias, residual, z, y, static_cast<cudaStream_t>(stream)); });
}

size_t dsv4v_linear_backward_workspace_size(const dsv4v_linear* layer) {
  Layer l;
  if (check_layer(layer, l) != DSV4V_OK) return 0;
  return std::max<size_t>(256, backward_layout(l, planning_sms()).total);
}

dsv4v_status dsv4v_linear_backward(const dsv4v_linear* layer, const void* x, const void* w, const void* z, const void* d_y, void* dx,
                                   void* dw, float* db, void* workspace, size_t ws_bytes, void* stream) {
  Layer l;
  const dsv4v_status st = check_layer(layer, l);
  if (st != DSV4V_OK) return st;
  const size_t in = l.bf16 ? 16 : 4;
  const bool act = l.act != DSV4V_ACT_NONE;
  if ((dw && !aligned_to(dw, l.es)) || (db && !aligned_to(db, 4)) || (dx && !aligned_to(dx, l.es))) return DSV4V_ERR_INVALID_ARG;
  if (l.rows > 0) {
    if (!d_y || !aligned_to(d_y, l.es) || (act && (!z || !aligned_to(z, l.es))) || (dx && (!w || !aligned_to(w, in))) ||
        (dw && (!x || !aligned_to(x, in))))
      return DSV4V_ERR_INVALID_ARG;
    if (dx && (dx == d_y || dx == w || dx == z || dx == x)) return DSV4V_ERR_INVALID_ARG;
    if (dw && (dw == x || dw == d_y || dw == z || dw == dx)) return DSV4V_ERR_INVALID_ARG;
  }
  if (dw && dw == w) return DSV4V_ERR_INVALID_ARG;  // without rows too, which clears dw
  int sms = 0;
  if (!query_device(&sms, nullptr)) return DSV4V_ERR_CUDA;
  const BackwardLayout bl = backward_layout(l, sms);
  if (!workspace || !aligned_to(workspace, 256) || ws_bytes < std::max<size_t>(256, bl.total)) return DSV4V_ERR_WORKSPACE;
  return guarded([&] {
    return backward(l, x, w, z, d_y, dx, dw, db, static_cast<uint8_t*>(workspace), bl, sms, static_cast<cudaStream_t>(stream));
  });
}

}  // extern "C"
