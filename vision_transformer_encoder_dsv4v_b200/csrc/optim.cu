// The optimizer end of a training step over a list of tensors: the global gradient norm and the
// AdamW step, with states in fp32 or in 8 bits.
//
// Both read every tensor once and do a handful of operations per element, so HBM bounds them.
// The tensor list travels in the kernel's parameters (the constant bank): no device copy of it to
// keep, to stage or to race with, and a captured launch holds its own.  The tensors are cut into
// chunks numbered through the list, and every CTA walks an equal, contiguous range of chunks: one
// search for the first chunk's tensor, then steps along the list.  Lists longer than a table are
// taken in several launches.
#include <cuda_fp8.h>
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "dsv4v.h"
#include "internal.h"

namespace dsv4v {

namespace {

constexpr int kThreads = 256;
constexpr int kParamBytes = 32000;  // of the 32,764 bytes that a kernel may take

// Elements i .. i + 7 of a bf16 or fp32 array, as fp32; `cnt` of them exist (the rest read as 0).
__device__ __forceinline__ void load8(const void* base, bool bf16, bool vec, int64_t i, int cnt, float (&v)[8]) {
  if (vec && cnt == 8) {
    if (bf16) {
      const uint4 q = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(base) + i);
      v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
      v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
    } else {
      const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(base) + i);
      const float4 a = p[0], b = p[1];
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    v[j] = 0.0f;
    if (j < cnt)
      v[j] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[i + j]) : static_cast<const float*>(base)[i + j];
  }
}

__device__ __forceinline__ void store8(void* base, bool bf16, bool vec, int64_t i, int cnt, const float (&v)[8]) {
  if (vec && cnt == 8) {
    if (bf16) {
      *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(base) + i) =
          make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
    } else {
      float4* p = reinterpret_cast<float4*>(static_cast<float*>(base) + i);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (j >= cnt) break;
    if (bf16) static_cast<__nv_bfloat16*>(base)[i + j] = __float2bfloat16_rn(v[j]);
    else static_cast<float*>(base)[i + j] = v[j];
  }
}

// Chunks [lo, hi) of CTA `b` of `g`.
__device__ __forceinline__ uint32_t chunk_begin(uint32_t b, uint32_t g, uint32_t chunks) {
  return static_cast<uint32_t>(static_cast<uint64_t>(b) * chunks / g);
}

// ---------------------------------------------------------------------------- gradient norm
constexpr int kNormChunk = kThreads * 8 * 4;  // elements
constexpr int kNormMaxCtas = 2048;            // partial sums of one launch

struct NormEntry {
  const void* data;
  int64_t n;
  uint32_t chunk0;  // number of this tensor's first chunk
  uint32_t flags;   // 1: bf16, 2: 16-byte aligned
};
constexpr int kNormCap = (kParamBytes - 64) / static_cast<int>(sizeof(NormEntry));
struct NormTable {
  double* partials;
  uint32_t chunks;
  int count;
  NormEntry e[kNormCap];
};

// Sum of squares of 8 values.  fp32 (relative error of a few 2^-24, which the outer fp64 sum
// averages out) unless the squares leave fp32's range, which a second look in fp64 covers: the
// norm holds for every finite gradient.
__device__ __forceinline__ double squares8(const float (&v)[8]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
  if (s > 1e-30f && s < 1e37f) return static_cast<double>(s);
  double d = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) d = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), d);
  return d;
}

// Sum over the block in a fixed order; thread 0 holds it.
template <int THREADS>
__device__ __forceinline__ double block_sum(double v) {
  __shared__ double warp_sum[THREADS / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
  if ((threadIdx.x & 31) == 0) warp_sum[threadIdx.x >> 5] = v;
  __syncthreads();
  double s = 0.0;
  if (threadIdx.x == 0)
    for (int w = 0; w < THREADS / 32; ++w) s += warp_sum[w];
  return s;
}

__global__ void __launch_bounds__(kThreads, 4) k_grad_norm(const __grid_constant__ NormTable t) {
  launch_dependents();
  grid_dependency_wait();
  const uint32_t c0 = chunk_begin(blockIdx.x, gridDim.x, t.chunks), c1 = chunk_begin(blockIdx.x + 1, gridDim.x, t.chunks);
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= c0) lo = mid;
    else hi = mid - 1;
  }
  double acc = 0.0;
  for (uint32_t c = c0; c < c1; ++c) {
    while (lo + 1 < t.count && t.e[lo + 1].chunk0 <= c) ++lo;
    const NormEntry& e = t.e[lo];
    const bool bf16 = e.flags & 1u, vec = e.flags & 2u;
    const int64_t i0 = static_cast<int64_t>(c - e.chunk0) * kNormChunk + threadIdx.x * 8;
    float v[4][8];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + u * kThreads * 8;
      load8(e.data, bf16, vec, i, static_cast<int>(max(int64_t(0), min(int64_t(8), e.n - i))), v[u]);
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) acc += squares8(v[u]);
  }
  const double s = block_sum<kThreads>(acc);
  if (threadIdx.x == 0) t.partials[blockIdx.x] = s;
}

// norm = sqrt of the partial sums' sum, in a fixed order.
__global__ void __launch_bounds__(kThreads) k_grad_norm_final(const double* partials, int n, float* out) {
  launch_dependents();
  grid_dependency_wait();
  double acc = 0.0;
  for (int i = threadIdx.x; i < n; i += kThreads) acc += partials[i];
  const double s = block_sum<kThreads>(acc);
  if (threadIdx.x == 0) *out = static_cast<float>(sqrt(s));
}

// ---------------------------------------------------------------------------- AdamW
// A warp takes 256 consecutive elements of a tensor, 8 a lane: one block of an 8-bit state, so
// that its largest magnitude is a warp reduction.
constexpr int kStateBlock = 256;
constexpr int kAdamChunk = kThreads * 8;

enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kState8 = 4, kVector = 8 };

struct AdamEntry {
  void* param;
  const void* grad;
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  int64_t n;
  double decay;
  uint32_t chunk0;
  uint32_t flags;
};
struct AdamArgs {
  double lr, beta1, beta2;
  float b1, c1, b2, c2, eps;  // beta, 1 - beta (rounded from fp64)
  float max_norm;
  int64_t step;
  const float* grad_norm;
  const float* lr_dev;
  const int64_t* step_dev;
};
constexpr int kAdamCap = (kParamBytes - 160) / static_cast<int>(sizeof(AdamEntry));
struct AdamTable {
  AdamArgs a;
  uint32_t chunks;
  int count;
  AdamEntry e[kAdamCap];
};

__device__ __forceinline__ double int_power(double b, int64_t t) {
  double r = 1.0;
  for (; t > 0; t >>= 1) {
    if (t & 1) r *= b;
    b *= b;
  }
  return r;
}

// Whether the step is taken: a gradient norm that is not finite skips it.
__device__ __forceinline__ bool step_taken(const float* grad_norm) {
  return !grad_norm || (__float_as_uint(*grad_norm) & 0x7f800000u) != 0x7f800000u;
}

// Biased exponent of the power-of-two scale of a block whose largest magnitude has the bits
// `top`: the smallest 2^e with top / 2^e <= 448 = 1.75 * 2^8, e >= -126.  A power of two makes the
// division exact, so only the rounding to e4m3 is lost, and costs no precision: e4m3 is a
// floating type that needs the block's range, not its exact maximum.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t top) {
  const int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 1));
}

// Largest finite magnitude over the warp's 256 values, as bits (bits of magnitudes order like
// the magnitudes).
__device__ __forceinline__ uint32_t warp_top(const float (&v)[8]) {
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t b = __float_as_uint(v[j]) & 0x7fffffffu;
    top = max(top, b < 0x7f800000u ? b : 0u);
  }
  return __reduce_max_sync(0xffffffffu, top);
}

__device__ __forceinline__ void decode8(uint2 codes, float scale, float (&v)[8]) {
  const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2(static_cast<__nv_fp8x2_storage_t>(w[h >> 1] >> (16 * (h & 1))), __NV_E4M3);
    const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
    v[2 * h] = f.x * scale;
    v[2 * h + 1] = f.y * scale;
  }
}

// Codes of v * inv, rounded to nearest even; what is not finite becomes the NaN code.
__device__ __forceinline__ uint2 encode8(const float (&v)[8], float inv) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float a = v[2 * h] * inv, b = v[2 * h + 1] * inv;
    a = (__float_as_uint(a) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : a;
    b = (__float_as_uint(b) & 0x7f800000u) == 0x7f800000u ? __uint_as_float(0x7fffffffu) : b;
    w[h >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3)) << (16 * (h & 1));
  }
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 load_codes(const void* base, bool vec, int64_t i, int cnt) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  if (vec && cnt == 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < cnt) w[j >> 2] |= static_cast<uint32_t>(p[j]) << (8 * (j & 3));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ void store_codes(void* base, bool vec, int64_t i, int cnt, uint2 c) {
  uint8_t* p = static_cast<uint8_t*>(base) + i;
  if (vec && cnt == 8) {
    *reinterpret_cast<uint2*>(p) = c;
    return;
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j < cnt) p[j] = static_cast<uint8_t>((j < 4 ? c.x : c.y) >> (8 * (j & 3)));
}

// One AdamW step of 8 elements a thread:
//   g' = g min(1, max_norm / norm);  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p = p (1 - lr decay) - (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps)
// m and v take each product and sum rounded by itself (no contraction): a block's scale then
// depends on the formula alone, not on how a compiler fuses it.
__global__ void __launch_bounds__(kThreads, 4) k_adamw(const __grid_constant__ AdamTable t) {
  grid_dependency_wait();
  const AdamArgs& a = t.a;
  __shared__ double s_lr;
  __shared__ float s_step_size, s_inv_root;
  if (!step_taken(a.grad_norm)) return;
  if (threadIdx.x == 0) {
    const double lr = a.lr_dev ? static_cast<double>(*a.lr_dev) : a.lr;
    const int64_t step = a.step_dev ? *a.step_dev + 1 : a.step;
    s_lr = lr;
    s_step_size = static_cast<float>(lr / (1.0 - int_power(a.beta1, step)));
    s_inv_root = static_cast<float>(1.0 / sqrt(1.0 - int_power(a.beta2, step)));
  }
  __syncthreads();
  const double lr = s_lr;
  const float step_size = s_step_size, inv_root = s_inv_root;
  float clip = 1.0f;
  if (a.grad_norm && a.max_norm > 0.0f) clip = fminf(1.0f, __fdiv_rn(a.max_norm, *a.grad_norm));
  const int lane = threadIdx.x & 31;

  const uint32_t c0 = chunk_begin(blockIdx.x, gridDim.x, t.chunks), c1 = chunk_begin(blockIdx.x + 1, gridDim.x, t.chunks);
  int lo = 0, hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= c0) lo = mid;
    else hi = mid - 1;
  }
  for (uint32_t c = c0; c < c1; ++c) {
    while (lo + 1 < t.count && t.e[lo + 1].chunk0 <= c) ++lo;
    const AdamEntry& e = t.e[lo];
    const bool vec = e.flags & kVector, s8 = e.flags & kState8;
    const int64_t i = static_cast<int64_t>(c - e.chunk0) * kAdamChunk + threadIdx.x * 8;
    if (i - lane * 8 >= e.n) continue;  // the whole warp lies behind the tensor's end
    const int cnt = static_cast<int>(max(int64_t(0), min(int64_t(8), e.n - i)));
    const int64_t block = i / kStateBlock;  // the same for the warp
    float g[8], p[8], m[8], v[8];
    load8(e.grad, e.flags & kGradBf16, vec, i, cnt, g);
    if (e.master) load8(e.master, false, vec, i, cnt, p);
    else load8(e.param, e.flags & kParamBf16, vec, i, cnt, p);
    if (s8) {
      const uint2 mc = load_codes(e.m, vec, i, cnt), vc = load_codes(e.v, vec, i, cnt);
      decode8(mc, e.m_scale[block], m);
      decode8(vc, e.v_scale[block], v);
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
    } else {
      load8(e.m, false, vec, i, cnt, m);
      load8(e.v, false, vec, i, cnt, v);
    }
    const float keep = static_cast<float>(1.0 - lr * e.decay);
    float root[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      const float gj = __fmul_rn(g[j], clip);
      m[j] = __fadd_rn(__fmul_rn(m[j], a.b1), __fmul_rn(gj, a.c1));
      v[j] = __fadd_rn(__fmul_rn(v[j], a.b2), __fmul_rn(__fmul_rn(gj, gj), a.c2));
      root[j] = __fsqrt_rn(v[j]);
      p[j] = __fsub_rn(__fmul_rn(p[j], keep), __fmul_rn(step_size, __fdiv_rn(m[j], __fadd_rn(__fmul_rn(root[j], inv_root), a.eps))));
    }
    store8(e.param, e.flags & kParamBf16, vec, i, cnt, p);
    if (e.master) store8(e.master, false, vec, i, cnt, p);
    if (s8) {
      const uint32_t m_top = warp_top(m), r_top = warp_top(root);
      const uint32_t me = scale_exponent(m_top), re = scale_exponent(r_top);
      const uint2 mc = encode8(m, m_top ? __uint_as_float((254u - me) << 23) : 1.0f);
      uint2 vc = encode8(root, r_top ? __uint_as_float((254u - re) << 23) : 1.0f);
      // A root above zero never becomes zero: m may still be large there, and m / eps would blow
      // the step up.
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        uint32_t& w = j < 4 ? vc.x : vc.y;
        if (root[j] > 0.0f && ((w >> (8 * (j & 3))) & 0x7fu) == 0) w |= 1u << (8 * (j & 3));
      }
      store_codes(e.m, vec, i, cnt, mc);
      store_codes(e.v, vec, i, cnt, vc);
      if (lane == 0) {
        e.m_scale[block] = m_top ? __uint_as_float(me << 23) : 0.0f;
        e.v_scale[block] = r_top ? __uint_as_float(re << 23) : 0.0f;
      }
    } else {
      store8(e.m, false, vec, i, cnt, m);
      store8(e.v, false, vec, i, cnt, v);
    }
  }
}

// Last launch of a step, without the dependent-launch attribute: it starts when every weight is
// written, so that a following call's early weight loads (which only wait for the kernel before
// them to begin) cannot meet a weight that is still being written.  It counts the step too.
__global__ void k_adamw_end(int64_t* step_dev, const float* grad_norm) {
  if (step_dev && step_taken(grad_norm)) ++*step_dev;
}

bool aligned_to(const void* p, size_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }

bool known_dtype(int d) { return d == DSV4V_F32 || d == DSV4V_BF16; }

uint32_t chunks_of(int64_t n, int chunk) { return static_cast<uint32_t>((n + chunk - 1) / chunk); }

// Elements of a whole list: keeps the chunk numbers of a table below 2^32.
constexpr int64_t kMaxElements = int64_t(1) << 40;

dsv4v_status check_grads(const dsv4v_grad* grads, int n_tensors) {
  if (n_tensors < 0 || (n_tensors > 0 && !grads)) return DSV4V_ERR_INVALID_ARG;
  int64_t left = kMaxElements;
  for (int i = 0; i < n_tensors; ++i) {
    const dsv4v_grad& g = grads[i];
    if (g.n < 0 || !known_dtype(g.dtype)) return DSV4V_ERR_INVALID_ARG;
    if (g.n > left) return DSV4V_ERR_UNSUPPORTED;
    left -= g.n;
    if (g.n > 0 && (!g.data || !aligned_to(g.data, g.dtype == DSV4V_BF16 ? 2 : 4))) return DSV4V_ERR_INVALID_ARG;
  }
  return DSV4V_OK;
}

dsv4v_status check_tensor(const dsv4v_adamw_tensor& t) {
  if (t.n < 0 || !known_dtype(t.param_dtype) || !known_dtype(t.grad_dtype) || (t.state_bits != 32 && t.state_bits != 8) ||
      !(t.weight_decay >= 0.0) || !std::isfinite(t.weight_decay))
    return DSV4V_ERR_INVALID_ARG;
  if (t.n == 0) return DSV4V_OK;
  if (!t.param || !t.grad || !t.exp_avg || !t.exp_avg_sq) return DSV4V_ERR_INVALID_ARG;
  if (!aligned_to(t.param, t.param_dtype == DSV4V_BF16 ? 2 : 4) || !aligned_to(t.grad, t.grad_dtype == DSV4V_BF16 ? 2 : 4))
    return DSV4V_ERR_INVALID_ARG;
  if (t.master && (t.param_dtype != DSV4V_BF16 || !aligned_to(t.master, 4))) return DSV4V_ERR_INVALID_ARG;
  if (t.state_bits == 8) {
    if (!t.exp_avg_scale || !t.exp_avg_sq_scale || !aligned_to(t.exp_avg_scale, 4) || !aligned_to(t.exp_avg_sq_scale, 4))
      return DSV4V_ERR_INVALID_ARG;
  } else if (t.exp_avg_scale || t.exp_avg_sq_scale || !aligned_to(t.exp_avg, 4) || !aligned_to(t.exp_avg_sq, 4)) {
    return DSV4V_ERR_INVALID_ARG;
  }
  return DSV4V_OK;
}

// Launches k_adamw for the tensors a table holds.
dsv4v_status launch_adamw(AdamTable& t, int sms, cudaStream_t s) {
  if (t.count == 0) return DSV4V_OK;
  const unsigned grid = std::min<unsigned>(t.chunks, 4u * static_cast<unsigned>(sms));
  return launch_pdl(k_adamw, dim3(grid), dim3(kThreads), 0, s, t) == cudaSuccess ? DSV4V_OK : DSV4V_ERR_CUDA;
}

}  // namespace

}  // namespace dsv4v

using namespace dsv4v;

extern "C" {

size_t dsv4v_grad_norm_workspace_size(int n_tensors) {
  if (n_tensors < 0) return 0;
  const size_t launches = std::max<size_t>(1, (static_cast<size_t>(n_tensors) + kNormCap - 1) / kNormCap);
  return launches * kNormMaxCtas * sizeof(double);
}

dsv4v_status dsv4v_grad_norm(const dsv4v_grad* grads, int n_tensors, float* norm_out, void* workspace, size_t ws_bytes,
                             void* stream) {
  const dsv4v_status st = check_grads(grads, n_tensors);
  if (st != DSV4V_OK) return st;
  if (!norm_out || !aligned_to(norm_out, 4)) return DSV4V_ERR_INVALID_ARG;
  if (!workspace || !aligned_to(workspace, 256) || ws_bytes < dsv4v_grad_norm_workspace_size(n_tensors))
    return DSV4V_ERR_WORKSPACE;
  int sms = 0;
  if (!query_device(&sms, nullptr)) return DSV4V_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  double* partials = static_cast<double*>(workspace);
  int used = 0;
  static thread_local NormTable t;
  for (int i = 0; i < n_tensors;) {
    t.partials = partials + used;
    t.chunks = 0;
    t.count = 0;
    for (; i < n_tensors && t.count < kNormCap; ++i) {
      const dsv4v_grad& g = grads[i];
      if (g.n == 0) continue;
      const uint32_t c = chunks_of(g.n, kNormChunk);
      t.e[t.count++] = NormEntry{g.data, g.n, t.chunks, (g.dtype == DSV4V_BF16 ? 1u : 0u) | (aligned_to(g.data, 16) ? 2u : 0u)};
      t.chunks += c;
    }
    if (t.count == 0) continue;
    const unsigned grid = std::min<unsigned>({t.chunks, 4u * static_cast<unsigned>(sms), static_cast<unsigned>(kNormMaxCtas)});
    if (launch_pdl(k_grad_norm, dim3(grid), dim3(kThreads), 0, s, t) != cudaSuccess) return DSV4V_ERR_CUDA;
    used += static_cast<int>(grid);
  }
  return launch_pdl(k_grad_norm_final, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(partials), used, norm_out) ==
                 cudaSuccess
             ? DSV4V_OK
             : DSV4V_ERR_CUDA;
}

dsv4v_status dsv4v_adamw_step(const dsv4v_adamw_config* cfg, const dsv4v_adamw_tensor* tensors, int n_tensors,
                              const float* grad_norm, const float* lr_dev, int64_t* step_dev, void* stream) {
  if (!cfg || n_tensors < 0 || (n_tensors > 0 && !tensors)) return DSV4V_ERR_INVALID_ARG;
  if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) || !(static_cast<float>(cfg->eps) > 0.0f) ||
      !std::isfinite(static_cast<float>(cfg->eps)) || !std::isfinite(cfg->lr) || !(cfg->max_grad_norm >= 0.0) ||
      !std::isfinite(static_cast<float>(cfg->max_grad_norm)) || (!step_dev && cfg->step < 1) || (cfg->max_grad_norm > 0.0 && !grad_norm))
    return DSV4V_ERR_INVALID_ARG;
  if ((grad_norm && !aligned_to(grad_norm, 4)) || (lr_dev && !aligned_to(lr_dev, 4)) || (step_dev && !aligned_to(step_dev, 8)))
    return DSV4V_ERR_INVALID_ARG;
  int64_t left = kMaxElements;
  for (int i = 0; i < n_tensors; ++i) {
    const dsv4v_status st = check_tensor(tensors[i]);
    if (st != DSV4V_OK) return st;
    if (tensors[i].n > left) return DSV4V_ERR_UNSUPPORTED;
    left -= tensors[i].n;
  }
  int sms = 0;
  if (!query_device(&sms, nullptr)) return DSV4V_ERR_CUDA;
  cudaStream_t s = static_cast<cudaStream_t>(stream);
  static thread_local AdamTable t;
  t.a.lr = cfg->lr;
  t.a.beta1 = cfg->beta1;
  t.a.beta2 = cfg->beta2;
  t.a.b1 = static_cast<float>(cfg->beta1);
  t.a.c1 = static_cast<float>(1.0 - cfg->beta1);
  t.a.b2 = static_cast<float>(cfg->beta2);
  t.a.c2 = static_cast<float>(1.0 - cfg->beta2);
  t.a.eps = static_cast<float>(cfg->eps);
  t.a.max_norm = static_cast<float>(cfg->max_grad_norm);
  t.a.step = cfg->step;
  t.a.grad_norm = grad_norm;
  t.a.lr_dev = lr_dev;
  t.a.step_dev = step_dev;
  for (int i = 0; i < n_tensors;) {
    t.chunks = 0;
    t.count = 0;
    for (; i < n_tensors && t.count < kAdamCap; ++i) {
      const dsv4v_adamw_tensor& x = tensors[i];
      if (x.n == 0) continue;
      const uint32_t c = chunks_of(x.n, kAdamChunk);
      const bool s8 = x.state_bits == 8;
      const size_t state_align = s8 ? 8 : 16;
      const bool vec = aligned_to(x.param, 16) && aligned_to(x.grad, 16) && (!x.master || aligned_to(x.master, 16)) &&
                       aligned_to(x.exp_avg, state_align) && aligned_to(x.exp_avg_sq, state_align);
      t.e[t.count++] = AdamEntry{x.param, x.grad, x.master, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale, x.exp_avg_sq_scale, x.n,
                                 x.weight_decay, t.chunks,
                                 (x.param_dtype == DSV4V_BF16 ? kParamBf16 : 0u) | (x.grad_dtype == DSV4V_BF16 ? kGradBf16 : 0u) |
                                     (s8 ? kState8 : 0u) | (vec ? kVector : 0u)};
      t.chunks += c;
    }
    const dsv4v_status st = launch_adamw(t, sms, s);
    if (st != DSV4V_OK) return st;
  }
  k_adamw_end<<<1, 1, 0, s>>>(step_dev, grad_norm);
  return cudaGetLastError() == cudaSuccess ? DSV4V_OK : DSV4V_ERR_CUDA;
}

}  // extern "C"
