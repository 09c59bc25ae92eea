// The optimizer end of a training step over a list of tensors: the global gradient norm and the
// AdamW step, with states in fp32 or in 8 bits.
//
// Both read every tensor once and do a handful of operations per element, so HBM bounds them.
// The tensor list travels in the kernel's parameters (the constant bank): no device copy of it to
// keep, to stage or to race with, and a captured launch holds its own.  The tensors are cut into
// chunks numbered through the list and dealt to the CTAs in turn, so that the many small or ragged
// tensors of a list do not gather in a few CTAs (contiguous ranges left the SMs idle for 30% of
// the time).  Lists longer than a table are taken in several launches.
#include <cuda_fp8.h>
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "dsv4v.h"
#include "internal.h"

namespace dsv4v {

namespace {

constexpr int kThreads = 256;
// Bytes of a table: nearly all of the 32,764 that a kernel may take or, for short lists, fewer,
// which a launch copies sooner (65 tensors: 10.2 us a call from the host, against 11.5 us).
constexpr int kParamBytes = 32000, kShortBytes = 8000;

// Elements i .. i + 7 of a bf16 or fp32 array, as fp32; `cnt` of them exist (the rest read as 0;
// with cnt <= 0, element i + cnt - 1 does).
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
  // Every load reads an element that exists, so that none waits for a branch.
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const int64_t at = i + min(j, cnt - 1);
    v[j] = bf16 ? __bfloat162float(static_cast<const __nv_bfloat16*>(base)[at]) : static_cast<const float*>(base)[at];
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    if (j >= cnt) v[j] = 0.0f;
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

// Tensor of chunk c, which lies at tensor `lo` or behind it.
template <class Table>
__device__ __forceinline__ int tensor_of(const Table& t, uint32_t c, int lo) {
  if (lo + 1 >= t.count || t.e[lo + 1].chunk0 > c) return lo;
  int hi = t.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (t.e[mid].chunk0 <= c) lo = mid;
    else hi = mid - 1;
  }
  return lo;
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
template <int BYTES>
struct NormTable {
  static constexpr int CAP = (BYTES - 64) / static_cast<int>(sizeof(NormEntry));
  double* partials;
  uint32_t chunks;
  int count;
  NormEntry e[CAP];
};
constexpr int kNormCap = NormTable<kParamBytes>::CAP;

// Sum of squares of eight values.  fp32 (eight roundings, at most 8 x 2^-24 of the sum however the
// values are made) unless the squares leave fp32's range, which a second look in fp64 covers: the norm
// holds for every finite gradient.
__device__ __forceinline__ double squares(const float (&v)[8]) {
  float s = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) s = fmaf(v[j], v[j], s);
  if (s > 1e-30f && s < 1e37f) return static_cast<double>(s);
  double d = 0.0;
#pragma unroll
  for (int j = 0; j < 8; ++j) d = fma(static_cast<double>(v[j]), static_cast<double>(v[j]), d);
  return d;
}

__device__ __forceinline__ void unpack8(const uint4& q, float (&v)[8]) {
  v[0] = bf16_lo(q.x), v[1] = bf16_hi(q.x), v[2] = bf16_lo(q.y), v[3] = bf16_hi(q.y);
  v[4] = bf16_lo(q.z), v[5] = bf16_hi(q.z), v[6] = bf16_lo(q.w), v[7] = bf16_hi(q.w);
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

// 64 bytes of a thread are in flight at a time for bf16 and 128 for fp32, 64 to 128 KB an SM, which
// is what hides HBM's latency.  A thread sums the same elements in the same order whether a chunk is
// whole, ragged or unaligned, so the norm does not depend on where the tensors lie.
template <int BYTES>
__global__ void __launch_bounds__(kThreads, 4) k_grad_norm(const __grid_constant__ NormTable<BYTES> t) {
  launch_dependents();
  grid_dependency_wait();
  double acc = 0.0;
  int lo = 0;
  for (uint32_t c = blockIdx.x; c < t.chunks; c += gridDim.x) {
    lo = tensor_of(t, c, lo);
    const NormEntry& e = t.e[lo];
    const bool bf16 = e.flags & 1u, vec = e.flags & 2u;
    const int64_t i0 = static_cast<int64_t>(c - e.chunk0) * kNormChunk;
    if (vec && i0 + kNormChunk <= e.n) {
      if (bf16) {
        const uint4* p = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(e.data) + i0) + threadIdx.x;
        uint4 q[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) q[u] = p[u * kThreads];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          float v[8];
          unpack8(q[u], v);
          acc += squares(v);
        }
      } else {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(e.data) + i0) + 2 * threadIdx.x;
        float4 q[8];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          q[2 * u] = p[2 * u * kThreads];
          q[2 * u + 1] = p[2 * u * kThreads + 1];
        }
#pragma unroll
        for (int u = 0; u < 8; u += 2) {
          const float v[8] = {q[u].x, q[u].y, q[u].z, q[u].w, q[u + 1].x, q[u + 1].y, q[u + 1].z, q[u + 1].w};
          acc += squares(v);
        }
      }
      continue;
    }
#pragma unroll 1
    for (int u = 0; u < 4; ++u) {
      const int64_t i = i0 + (u * kThreads + threadIdx.x) * 8;
      if (i >= e.n) break;
      float v[8];
      load8(e.data, bf16, vec, i, static_cast<int>(min(int64_t(8), e.n - i)), v);
      acc += squares(v);
    }
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

enum : uint32_t { kParamBf16 = 1, kGradBf16 = 2, kState8 = 4, kMaster = 8, kVector = 16, kStochastic = 32, kIndexShift = 8 };

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
  uint32_t flags;  // the tensor's place in the call's list from bit kIndexShift on
};
struct AdamArgs {
  double lr, beta1, beta2;
  int64_t step;
  float step_size, inv_root;  // lr / (1 - beta1^step), 1 / sqrt(1 - beta2^step)
  float b1, c1, b2, c2, eps;  // beta, 1 - beta (rounded from fp64)
  float max_norm;
  const float* grad_norm;
  const float* lr_dev;
  const int64_t* step_dev;
};
template <int BYTES>
struct AdamTable {
  static constexpr int CAP = (BYTES - 160) / static_cast<int>(sizeof(AdamEntry));
  AdamArgs a;
  uint32_t chunks;
  int count;
  AdamEntry e[CAP];
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
// division exact, so that a value changes by its rounding to e4m3 alone.
__device__ __forceinline__ uint32_t scale_exponent(uint32_t top) {
  const int e = static_cast<int>(top >> 23) - 8 + ((top & 0x7fffffu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 1));
}

// Largest magnitude over the warp's 256 values, as bits (bits of magnitudes order like the
// magnitudes); NaN does not count, infinity does unless `finite`.
__device__ __forceinline__ uint32_t warp_top(const float (&v)[8], bool finite) {
  float top = 0.0f;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float x = fabsf(v[j]);
    top = fmaxf(top, finite && x > 3.4028235e38f ? 0.0f : x);
  }
  return __reduce_max_sync(0xffffffffu, __float_as_uint(top));
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

// Codes of q (at most 448 in magnitude, or NaN), rounded to nearest even.
__device__ __forceinline__ uint2 encode8(const float (&q)[8]) {
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int h = 0; h < 4; ++h)
    w[h >> 1] |= static_cast<uint32_t>(__nv_cvt_float2_to_fp8x2(make_float2(q[2 * h], q[2 * h + 1]), __NV_SATFINITE, __NV_E4M3))
                 << (16 * (h & 1));
  return make_uint2(w[0], w[1]);
}

__device__ __forceinline__ uint2 load_codes(const void* base, bool vec, int64_t i, int cnt) {
  const uint8_t* p = static_cast<const uint8_t*>(base) + i;
  if (vec && cnt == 8) return *reinterpret_cast<const uint2*>(p);
  uint32_t w[2] = {0, 0};
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const uint32_t code = p[min(j, cnt - 1)];
    w[j >> 2] |= (j < cnt ? code : 0u) << (8 * (j & 3));
  }
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

__device__ __forceinline__ float sqrt_approx(float x) {
  float y;
  asm("sqrt.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct AdamScalars {
  float b1, c1, b2, c2, eps, clip, step_size, inv_root;
};

// Random words of a counter and a key: Philox 4x32 (Salmon, Moraes, Dror and Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011) of seven rounds, the number their tests of randomness ask for.
__device__ __forceinline__ void philox(uint4& c, uint32_t k0, uint32_t k1) {
#pragma unroll
  for (int r = 0; r < 7; ++r) {
    const uint64_t a = static_cast<uint64_t>(0xD2511F53u) * c.x, b = static_cast<uint64_t>(0xCD9E8D57u) * c.z;
    c = make_uint4(static_cast<uint32_t>(b >> 32) ^ c.y ^ k0, static_cast<uint32_t>(b),
                   static_cast<uint32_t>(a >> 32) ^ c.w ^ k1, static_cast<uint32_t>(a));
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
}

// Step of e4m3 at x >= 0 (2^-9 below 2^-6), and its inverse.
__device__ __forceinline__ float code_step(float x, float& inverse) {
  const uint32_t e = max(__float_as_uint(x) >> 23, 121u) - 3u;
  inverse = __uint_as_float((254u - e) << 23);
  return __uint_as_float(e << 23);
}

// One of the two e4m3 values around q, such that the expectation is q.
__device__ __forceinline__ float round_value(float q, uint32_t word) {
  float inv;
  const float step = code_step(fabsf(q), inv), t = fabsf(q) * inv, k = floorf(t);
  const float u = static_cast<float>(word >> 8) * 5.9604644775390625e-8f;  // 24 bits
  return copysignf((u < t - k ? k + 1.0f : k) * step, q);
}

// One of the two e4m3 values around root = sqrt(x) (approximately), such that the expectation of its
// square is x: it is the square that goes on as a moving average.
__device__ __forceinline__ float round_root(float x, float root, uint32_t word) {
  float inv;
  const float step = code_step(root, inv), t = x * inv * inv;
  float k = floorf(root * inv);
  if (t < k * k) k -= 1.0f;  // the root's own error crossed a whole step
  if (t >= (k + 1.0f) * (k + 1.0f)) k += 1.0f;
  const float u = static_cast<float>(word >> 8) * 5.9604644775390625e-8f;
  return (u * fmaf(2.0f, k, 1.0f) < fmaf(-k, k, t) ? k + 1.0f : k) * step;
}

// One AdamW step of the 8 elements that a thread holds:
//   g' = g min(1, max_norm / norm);  m = b1 m + (1 - b1) g';  v = b2 v + (1 - b2) g'^2
//   p = p - (lr decay p + (lr / (1 - b1^t)) m / (sqrt(v) / sqrt(1 - b2^t) + eps))
// The decay joins the update before p is rounded: as a factor 1 - lr decay it would come in steps of
// 2^-24, and not at all below 3e-8, where the ends of a schedule take it.
// m and v take each product and sum rounded by itself (no contraction): a block's scale then
// depends on the formula alone, not on how a compiler fuses it.  The update's root and quotient
// come from the MUFU pipe, off by 2^-23 of the update, which leaves the 8-bit step's 60 instructions an
// element within HBM's time.
__device__ __forceinline__ void adam8(const AdamScalars& a, float decay, const float (&g)[8], float (&p)[8], float (&m)[8],
                                      float (&v)[8], float (&root)[8]) {
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float gj = __fmul_rn(g[j], a.clip);
    m[j] = __fadd_rn(__fmul_rn(m[j], a.b1), __fmul_rn(gj, a.c1));
    v[j] = __fadd_rn(__fmul_rn(v[j], a.b2), __fmul_rn(__fmul_rn(gj, gj), a.c2));
    root[j] = sqrt_approx(v[j]);
    const float update = a.step_size * m[j] * rcp_approx(fmaf(root[j], a.inv_root, a.eps));
    p[j] -= fabsf(p[j]) <= 3.4028235e38f ? fmaf(decay, p[j], update) : update;  // a weight that masks by its infinity keeps it
  }
}

// Codes and scales of a block's new moments.  Rounded to nearest, a moment moves only by more than half a
// step of its code, 3 to 6 %: an average that takes less than that of each gradient stands still.  Rounded
// stochastically it moves as the formula does on average, by draws that the step, the tensor and the
// element `i` number: a repeated call repeats its codes.  The draws and their comparisons are about 50
// instructions an element (eight blocks 302 -> 457 us, bound by issue), so that they have a kernel of their
// own (STOCHASTIC) and the others keep their registers.
template <bool STOCHASTIC>
__device__ __forceinline__ void adam_codes(const AdamEntry& e, int64_t step, int64_t i, const float (&m)[8], const float (&v)[8],
                                           const float (&root)[8], uint2& mc, uint2& vc, float& m_scale, float& v_scale) {
  uint32_t m_top = warp_top(m, false), v_top = warp_top(v, false);
  const bool wild = max(m_top, v_top) >= 0x7f800000u;  // an infinity in the block, for the whole warp
  if (wild) {
    m_top = warp_top(m, true);
    v_top = warp_top(v, true);
  }
  const uint32_t r_top = __float_as_uint(__fsqrt_rn(__uint_as_float(v_top)));
  const uint32_t me = scale_exponent(m_top), re = scale_exponent(r_top);
  m_scale = m_top ? __uint_as_float(me << 23) : 0.0f;
  v_scale = r_top ? __uint_as_float(re << 23) : 0.0f;
  const float m_inv = m_top ? __uint_as_float((254u - me) << 23) : 1.0f, r_inv = r_top ? __uint_as_float((254u - re) << 23) : 1.0f;
  float qm[8], qr[8];
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    qm[j] = m[j] * m_inv;
    qr[j] = root[j] * r_inv;
  }
  if (STOCHASTIC && (e.flags & kStochastic)) {
#pragma unroll
    for (int c = 0; c < 4; ++c) {  // the words of elements 2c and 2c + 1
      const uint64_t group = static_cast<uint64_t>(i) / 8;
      uint4 w = make_uint4(static_cast<uint32_t>(group), static_cast<uint32_t>(group >> 32) << 2 | c, static_cast<uint32_t>(step),
                           static_cast<uint32_t>(step >> 32));
      philox(w, e.flags >> kIndexShift, 0u);
      qm[2 * c] = round_value(qm[2 * c], w.x);
      qr[2 * c] = round_root(v[2 * c] * r_inv * r_inv, qr[2 * c], w.y);
      qm[2 * c + 1] = round_value(qm[2 * c + 1], w.z);
      qr[2 * c + 1] = round_root(v[2 * c + 1] * r_inv * r_inv, qr[2 * c + 1], w.w);
    }
  }
#pragma unroll
  for (int j = 0; j < 8; ++j)
    // A root above zero never becomes zero: m may still be large there, and m / eps would blow the
    // step up.
    if (v[j] > 0.0f && qr[j] < 0.001953125f) qr[j] = 0.001953125f;
  if (wild) {
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      if (fabsf(m[j]) > 3.4028235e38f) qm[j] = __uint_as_float(0x7fffffffu);
      if (v[j] > 3.4028235e38f) qr[j] = __uint_as_float(0x7fffffffu);
    }
  }
  mc = encode8(qm);
  vc = encode8(qr);
}

// The usual case, 8 elements that exist behind aligned pointers.  The types are template
// parameters, so that all loads are issued before the first of them is waited for.
template <uint32_t KIND, bool STOCHASTIC>
__device__ __forceinline__ void adam_whole(const AdamEntry& e, const AdamScalars& a, float decay, int64_t step, int64_t i, int lane) {
  constexpr bool PB = KIND & kParamBf16, GB = KIND & kGradBf16, S8 = KIND & kState8, MASTER = KIND & kMaster;
  float g[8], p[8], m[8], v[8], root[8];
  uint2 mc, vc;
  float m_scale, v_scale;
  load8(e.grad, GB, true, i, 8, g);
  if constexpr (MASTER) load8(e.master, false, true, i, 8, p);
  else load8(e.param, PB, true, i, 8, p);
  if constexpr (S8) {
    mc = load_codes(e.m, true, i, 8);
    vc = load_codes(e.v, true, i, 8);
    m_scale = e.m_scale[i / kStateBlock];
    v_scale = e.v_scale[i / kStateBlock];
    decode8(mc, m_scale, m);
    decode8(vc, v_scale, v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
  } else {
    load8(e.m, false, true, i, 8, m);
    load8(e.v, false, true, i, 8, v);
  }
  adam8(a, decay, g, p, m, v, root);
  store8(e.param, PB, true, i, 8, p);
  if constexpr (MASTER) store8(e.master, false, true, i, 8, p);
  if constexpr (S8) {
    adam_codes<STOCHASTIC>(e, step, i, m, v, root, mc, vc, m_scale, v_scale);
    store_codes(e.m, true, i, 8, mc);
    store_codes(e.v, true, i, 8, vc);
    if (lane == 0) {
      e.m_scale[i / kStateBlock] = m_scale;
      e.v_scale[i / kStateBlock] = v_scale;
    }
  } else {
    store8(e.m, false, true, i, 8, m);
    store8(e.v, false, true, i, 8, v);
  }
}

// A tensor's ragged end, and tensors that are not aligned: any types, `cnt` elements (at most 8; for
// the lanes behind the end, 0 or less).
template <bool STOCHASTIC>
__device__ __noinline__ void adam_ragged(const AdamEntry& e, const AdamScalars& a, float decay, int64_t step, int64_t i, int cnt, int lane) {
  const bool vec = e.flags & kVector, s8 = e.flags & kState8, pb = e.flags & kParamBf16;
  const int64_t block = (i - lane * 8) / kStateBlock;
  float g[8], p[8], m[8], v[8], root[8];
  load8(e.grad, e.flags & kGradBf16, vec, i, cnt, g);
  if (e.master) load8(e.master, false, vec, i, cnt, p);
  else load8(e.param, pb, vec, i, cnt, p);
  if (s8) {
    decode8(load_codes(e.m, vec, i, cnt), e.m_scale[block], m);
    decode8(load_codes(e.v, vec, i, cnt), e.v_scale[block], v);
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = __fmul_rn(v[j], v[j]);
  } else {
    load8(e.m, false, vec, i, cnt, m);
    load8(e.v, false, vec, i, cnt, v);
  }
  adam8(a, decay, g, p, m, v, root);
  store8(e.param, pb, vec, i, cnt, p);
  if (e.master) store8(e.master, false, vec, i, cnt, p);
  if (s8) {
    uint2 mc, vc;
    float m_scale, v_scale;
    adam_codes<STOCHASTIC>(e, step, i, m, v, root, mc, vc, m_scale, v_scale);
    __syncwarp();  // every lane has read the block's old scales
    store_codes(e.m, vec, i, cnt, mc);
    store_codes(e.v, vec, i, cnt, vc);
    if (lane == 0) {
      e.m_scale[block] = m_scale;
      e.v_scale[block] = v_scale;
    }
  } else {
    store8(e.m, false, vec, i, cnt, m);
    store8(e.v, false, vec, i, cnt, v);
  }
}

// A CTA takes one chunk: CTAs that start in the chunks' order sweep each array front to back, which
// HBM rewards (427 us for 103 M bf16 weights with fp32 masters and states, 3.08 GB, back to back on the same
// arrays, 433 to 468 us on three sets of arrays in turn, by where they lie; a persistent grid that strides
// over the chunks took 536 us, contiguous ranges 527 us).
template <int BYTES, bool STOCHASTIC>
__global__ void __launch_bounds__(kThreads, 4) k_adamw(const __grid_constant__ AdamTable<BYTES> t) {
  grid_dependency_wait();
  if (!step_taken(t.a.grad_norm)) return;
  double lr = t.a.lr;
  float step_size = t.a.step_size, inv_root = t.a.inv_root;
  int64_t step = STOCHASTIC ? t.a.step : 0;
  if (t.a.lr_dev || t.a.step_dev) {  // the schedule lies on the device
    __shared__ double s_lr;
    __shared__ float s_step_size, s_inv_root;
    __shared__ int64_t s_step;
    if (threadIdx.x == 0) {
      if (t.a.lr_dev) lr = static_cast<double>(*t.a.lr_dev);
      const int64_t step = t.a.step_dev ? *t.a.step_dev + 1 : t.a.step;
      if constexpr (STOCHASTIC) s_step = step;
      s_lr = lr;
      s_step_size = static_cast<float>(lr / (1.0 - int_power(t.a.beta1, step)));
      s_inv_root = static_cast<float>(1.0 / sqrt(1.0 - int_power(t.a.beta2, step)));
    }
    __syncthreads();
    lr = s_lr;
    step_size = s_step_size;
    inv_root = s_inv_root;
    if constexpr (STOCHASTIC) step = s_step;
  }
  AdamScalars a{t.a.b1, t.a.c1, t.a.b2, t.a.c2, t.a.eps, 1.0f, step_size, inv_root};
  if (t.a.grad_norm && t.a.max_norm > 0.0f) a.clip = fminf(1.0f, __fdiv_rn(t.a.max_norm, *t.a.grad_norm));
  const int lane = threadIdx.x & 31;

  const uint32_t c = blockIdx.x;
  const AdamEntry& e = t.e[tensor_of(t, c, 0)];
  const float decay = static_cast<float>(lr * e.decay);
  const int64_t i = static_cast<int64_t>(c - e.chunk0) * kAdamChunk + threadIdx.x * 8;
  const int64_t end = i - lane * 8 + 256;  // of the warp's elements
  if (end <= e.n && (e.flags & kVector)) {
    switch (e.flags & 15u) {
      case 0: adam_whole<0, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kParamBf16: adam_whole<kParamBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kGradBf16: adam_whole<kGradBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kParamBf16 | kGradBf16: adam_whole<kParamBf16 | kGradBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kState8: adam_whole<kState8, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kState8 | kParamBf16: adam_whole<kState8 | kParamBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kState8 | kGradBf16: adam_whole<kState8 | kGradBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kState8 | kParamBf16 | kGradBf16: adam_whole<kState8 | kParamBf16 | kGradBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kMaster | kParamBf16: adam_whole<kMaster | kParamBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kMaster | kParamBf16 | kGradBf16: adam_whole<kMaster | kParamBf16 | kGradBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      case kMaster | kState8 | kParamBf16: adam_whole<kMaster | kState8 | kParamBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
      default: adam_whole<kMaster | kState8 | kParamBf16 | kGradBf16, STOCHASTIC>(e, a, decay, step, i, lane); break;
    }
  } else if (end - 256 < e.n) {
    adam_ragged<STOCHASTIC>(e, a, decay, step, i, static_cast<int>(min(int64_t(8), e.n - i)), lane);
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
  if (t.state_rounding != DSV4V_ROUND_NEAREST && (t.state_rounding != DSV4V_ROUND_STOCHASTIC || t.state_bits != 8))
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

// Takes tensors [i, n) into one table and launches it; returns the first tensor not taken, or -1.
template <int BYTES>
int launch_norm(const dsv4v_grad* grads, int i, int n, double* partials, int sms, cudaStream_t s, int* used) {
  static thread_local NormTable<BYTES> t;
  t.partials = partials + *used;
  t.chunks = 0;
  t.count = 0;
  for (; i < n && t.count < t.CAP; ++i) {
    const dsv4v_grad& g = grads[i];
    if (g.n == 0) continue;
    t.e[t.count++] = NormEntry{g.data, g.n, t.chunks, (g.dtype == DSV4V_BF16 ? 1u : 0u) | (aligned_to(g.data, 16) ? 2u : 0u)};
    t.chunks += chunks_of(g.n, kNormChunk);
  }
  if (t.count == 0) return i;
  const unsigned grid = std::min<unsigned>({t.chunks, 4u * static_cast<unsigned>(sms), static_cast<unsigned>(kNormMaxCtas)});
  if (launch_pdl(k_grad_norm<BYTES>, dim3(grid), dim3(kThreads), 0, s, t) != cudaSuccess) return -1;
  *used += static_cast<int>(grid);
  return i;
}

template <int BYTES>
int launch_adamw(const AdamArgs& args, const dsv4v_adamw_tensor* tensors, int i, int n, int sms, cudaStream_t s) {
  static thread_local AdamTable<BYTES> t;
  t.a = args;
  t.chunks = 0;
  t.count = 0;
  bool stochastic = false;
  for (; i < n && t.count < t.CAP; ++i) {
    const dsv4v_adamw_tensor& x = tensors[i];
    if (x.n == 0) continue;
    stochastic |= x.state_rounding == DSV4V_ROUND_STOCHASTIC;
    const bool s8 = x.state_bits == 8;
    const size_t state_align = s8 ? 8 : 16;
    const bool vec = aligned_to(x.param, 16) && aligned_to(x.grad, 16) && (!x.master || aligned_to(x.master, 16)) &&
                     aligned_to(x.exp_avg, state_align) && aligned_to(x.exp_avg_sq, state_align);
    t.e[t.count++] = AdamEntry{x.param, x.grad, x.master, x.exp_avg, x.exp_avg_sq, x.exp_avg_scale, x.exp_avg_sq_scale, x.n,
                               x.weight_decay, t.chunks,
                               (x.param_dtype == DSV4V_BF16 ? kParamBf16 : 0u) | (x.grad_dtype == DSV4V_BF16 ? kGradBf16 : 0u) |
                                   (s8 ? kState8 : 0u) | (x.master ? kMaster : 0u) | (vec ? kVector : 0u) |
                                   (x.state_rounding == DSV4V_ROUND_STOCHASTIC ? kStochastic : 0u) |
                                   static_cast<uint32_t>(i) << kIndexShift};
    t.chunks += chunks_of(x.n, kAdamChunk);
  }
  if (t.count == 0) return i;
  const auto kernel = stochastic ? k_adamw<BYTES, true> : k_adamw<BYTES, false>;
  return launch_pdl(kernel, dim3(t.chunks), dim3(kThreads), 0, s, t) == cudaSuccess ? i : -1;
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
  for (int i = 0; i < n_tensors;) {
    i = n_tensors - i <= NormTable<kShortBytes>::CAP ? launch_norm<kShortBytes>(grads, i, n_tensors, partials, sms, s, &used)
                                                     : launch_norm<kParamBytes>(grads, i, n_tensors, partials, sms, s, &used);
    if (i < 0) return DSV4V_ERR_CUDA;
  }
  return launch_pdl(k_grad_norm_final, dim3(1), dim3(kThreads), 0, s, static_cast<const double*>(partials), used, norm_out) ==
                 cudaSuccess
             ? DSV4V_OK
             : DSV4V_ERR_CUDA;
}

dsv4v_status dsv4v_adamw_step(const dsv4v_adamw_config* cfg, const dsv4v_adamw_tensor* tensors, int n_tensors,
                              const float* grad_norm, const float* lr_dev, int64_t* step_dev, void* stream) {
  if (!cfg || n_tensors < 0 || (n_tensors > 0 && !tensors)) return DSV4V_ERR_INVALID_ARG;
  if (!(cfg->beta1 >= 0.0 && cfg->beta1 < 1.0) || !(cfg->beta2 >= 0.0 && cfg->beta2 < 1.0) || !(static_cast<float>(cfg->eps) >= 1.17549435e-38f) ||
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
  AdamArgs a{};
  a.lr = cfg->lr;
  a.beta1 = cfg->beta1;
  a.beta2 = cfg->beta2;
  a.step = cfg->step;
  if (!step_dev) {
    a.step_size = static_cast<float>(cfg->lr / (1.0 - std::pow(cfg->beta1, static_cast<double>(cfg->step))));
    a.inv_root = static_cast<float>(1.0 / std::sqrt(1.0 - std::pow(cfg->beta2, static_cast<double>(cfg->step))));
  }
  a.b1 = static_cast<float>(cfg->beta1);
  a.c1 = static_cast<float>(1.0 - cfg->beta1);
  a.b2 = static_cast<float>(cfg->beta2);
  a.c2 = static_cast<float>(1.0 - cfg->beta2);
  a.eps = static_cast<float>(cfg->eps);
  a.max_norm = static_cast<float>(cfg->max_grad_norm);
  a.grad_norm = grad_norm;
  a.lr_dev = lr_dev;
  a.step_dev = step_dev;
  for (int i = 0; i < n_tensors;) {
    i = n_tensors - i <= AdamTable<kShortBytes>::CAP ? launch_adamw<kShortBytes>(a, tensors, i, n_tensors, sms, s)
                                                     : launch_adamw<kParamBytes>(a, tensors, i, n_tensors, sms, s);
    if (i < 0) return DSV4V_ERR_CUDA;
  }
  return launch_plain(k_adamw_end, dim3(1), dim3(1), 0, s, step_dev, grad_norm) == cudaSuccess ? DSV4V_OK : DSV4V_ERR_CUDA;
}

}  // extern "C"
