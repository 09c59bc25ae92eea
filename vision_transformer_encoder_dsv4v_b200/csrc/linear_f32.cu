// The Linear layer's fp32 products on the bf16 tensor cores.
//
// A value is the sum of three bf16, x = x0 + x1 + x2 with |x1| <= 2^-8 |x| and |x2| <= 2^-16 |x| (8 bits
// of its mantissa each).  Both operands are split as 2^16 x, whose last bit is at least bf16's least value
// (2^-133): the three parts are then exact down to fp32's own least value, and the sums are scaled back.
// Of the nine products of two values the six largest are formed,
//   a b = a0 b0 + (a0 b1 + a1 b0) + (a0 b2 + a1 b1 + a2 b0) + O(2^-25 |a b|),
// in three MMAs, because the parts of B lie behind one another as more columns: a0 meets b0, b1 and
// b2, a1 meets b0 and b1, a2 meets b0.  The tensor core truncates as it accumulates (2^-23 of the sum
// an addition): the large products have columns of their own, and every 256 of the contraction all of
// them are added up in fp32 registers.  The result is about as far from the exact one as an fp32 dot
// product (2e-7), at 3 bf16 MMAs of 64, 128 and 192 columns in the place of 64 columns of FMAs: 777 x
// 588 -> 1001 takes 20 us (ten stages are 12 of them), 22.5 us with bias, GELU and residual, where 4 x 4-output
// FMA tiles took 46 us, bound by shared-memory reads.
//
// Roles (544 threads): warps 0 to 15 load fp32, split it and write the parts into a 3-stage ring
// (K-major, 128-byte swizzle, transposing where the contraction is not contiguous), and add up the
// accumulators, 16 columns each; warp 16 issues the MMAs.  All store the 128 x 64 tile at the end.
// A stage takes 1.2 us: about 390 instructions a thread, and 220 KB through shared memory and L1 (parts
// stored 74, read by the MMAs 98, loads 49); the MMAs alone need half of that.  Where there are fewer
// tiles than SMs, two to eight CTAs of a cluster share one, each with a part of the contraction; a
// rank stores its share of the rows and fetches the others' sums through distributed shared memory,
// in rank order.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "linear.h"

namespace dsv4v {

namespace {

constexpr int TM = 128, TN = 64, TK = 64;
constexpr int kConvert = 512, kThreads = kConvert + 32;
constexpr int kStages = 3;
constexpr int kFlush = 4;  // stages whose products share an accumulator: 256 of the contraction
constexpr int kABytes = TM * TK * 2, kBBytes = TN * TK * 2;
constexpr int kStageBytes = 3 * (kABytes + kBBytes);
constexpr int kSmem = 1024 + kStages * kStageBytes + 256;
constexpr int kAccCols = 3 * TN;  // a0 b0 | a0 b1 + a1 b0 + a2 b0 | a0 b2 + a1 b1
constexpr int kSumLd = TN + 1;
constexpr int kSumRows = TM + 32;  // with the rows that an unrolled read may touch behind the tile
static_assert(kSumRows * kSumLd * 4 <= kStages * kStageBytes, "the sums have to fit the ring");

constexpr float kScale = 65536.0f, kUnscale = 1.0f / (kScale * kScale);
constexpr float kLargest = 1e37f;  // of a sum that is taken as it is: far below the end of the accumulators' range

// bf16 parts of eight values times kScale, 16 bytes each.  A value that is not finite, or (from 2^111 on)
// whose multiple rounds to a bf16 infinity, gives parts that are not finite, and so are the sums that it
// enters: they are formed again in fp32 (see store_column_plain).
__device__ __forceinline__ void split8(const float (&x)[8], uint4 (&out)[3]) {
  uint32_t w[3][4];
#pragma unroll
  for (int h = 0; h < 4; ++h) {
    float a, b;
    const uint64_t scaled = mul2(pk2(x[2 * h], x[2 * h + 1]), pk2(kScale, kScale));
    upk2(scaled, a, b);
    w[0][h] = pack_bf16x2(a, b);
    const uint64_t r = sub2(scaled, bf16x2_f2(w[0][h]));
    upk2(r, a, b);
    w[1][h] = pack_bf16x2(a, b);
    upk2(sub2(r, bf16x2_f2(w[1][h])), a, b);
    w[2][h] = pack_bf16x2(a, b);
  }
#pragma unroll
  for (int q = 0; q < 3; ++q) out[q] = make_uint4(w[q][0], w[q][1], w[q][2], w[q][3]);
}

// A thread's share of an operand's ROWS x 64 part of a stage, in pieces of one row and eight
// consecutive contraction indices.  A thread's pieces are 64 rows (or, MN-major, 512 / ROWS pieces of
// the contraction) apart.
template <int ROWS, bool K_FAST>
struct Share {
  static constexpr int PIECES = ROWS * 8 / kConvert;
  const float* at;  // the first element of piece 0 in the next stage
  int64_t ld;
  bool vec, in[PIECES];  // 16-byte loads; rows that exist
  float x[PIECES][8];

  static __device__ __forceinline__ int row(int j) {
    const int t = static_cast<int>(threadIdx.x);
    return K_FAST ? t / 8 + kConvert / 8 * j : t % ROWS;
  }
  static __device__ __forceinline__ int piece(int j) {
    const int t = static_cast<int>(threadIdx.x);
    return K_FAST ? t % 8 : t / ROWS + kConvert / ROWS * j;
  }
  // Rows i0 .. of n_i, contraction indices from k0 on.
  __device__ __forceinline__ Share(const float* a, int64_t ld_, int64_t i0, int64_t n_i, int64_t k0) : ld(ld_) {
    vec = (reinterpret_cast<uintptr_t>(a) & 15) == 0 && ld % 4 == 0;
    const int64_t i = i0 + row(0), k = k0 + piece(0) * 8;
    at = a + (K_FAST ? i * ld + k : k * ld + i);
#pragma unroll
    for (int j = 0; j < PIECES; ++j) in[j] = i0 + row(j) < n_i;
  }
  // Starts loading piece j of the next stage, which `left` indices of the contraction remain for.
  __device__ __forceinline__ void load(int j, int left) {
    const float* p = at + (K_FAST ? kConvert / 8 : kConvert / ROWS * 8) * j * ld;
    left = in[j] ? left - piece(j) * 8 : 0;
    if (left >= 8 && (!K_FAST || vec)) {
      if constexpr (K_FAST) {
        const float4 lo = reinterpret_cast<const float4*>(p)[0], hi = reinterpret_cast<const float4*>(p)[1];
        x[j][0] = lo.x, x[j][1] = lo.y, x[j][2] = lo.z, x[j][3] = lo.w, x[j][4] = hi.x, x[j][5] = hi.y, x[j][6] = hi.z, x[j][7] = hi.w;
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) x[j][e] = p[e * ld];
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) x[j][e] = e < left ? p[K_FAST ? e : e * ld] : 0.0f;
    }
  }
  __device__ __forceinline__ void advance() { at += K_FAST ? TK : TK * ld; }
  // The piece's parts into the operand's three tiles.
  __device__ __forceinline__ void store(int j, uint8_t* tiles) const {
    uint4 parts[3];
    split8(x[j], parts);
    const int r = row(j);
    uint8_t* to = tiles + r * 128 + ((piece(j) ^ (r & 7)) << 4);
#pragma unroll
    for (int q = 0; q < 3; ++q) *reinterpret_cast<uint4*>(to + q * ROWS * TK * 2) = parts[q];
  }
};

// ---------------------------------------------------------------------------- epilogue
__device__ __forceinline__ float activate(float v, int act) {
  if (act == DSV4V_ACT_GELU) return 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
  return act == DSV4V_ACT_SILU ? v / (1.0f + expf(-v)) : v;
}

// Stores rows lr, lr + 8, .. below r1 of one column of a tile: y, z and res point at row lr, `sum` at
// its sum (KS ranks: in every rank's shared memory).  Four rows at a time, whose reads are then in
// flight together.
template <int KS>
__device__ __forceinline__ void store_column(const EpilogueF32& e, int lr, int r1, const float* sum, float bias, float* y,
                                             const float* res, float* z) {
  constexpr int STEP = kConvert / TN, U = 4;
  for (; lr < r1; lr += STEP * U, sum += STEP * U * kSumLd) {
    float v[U], add[U] = {0, 0, 0, 0};
    if constexpr (KS == 1) {
#pragma unroll
      for (int u = 0; u < U; ++u) v[u] = sum[STEP * u * kSumLd];  // rows behind the end hold sums too
    } else {
      float q[KS][U];
#pragma unroll
      for (int k = 0; k < KS; ++k) {
        const uint32_t peer = mapa_shared(smem_u32(sum), static_cast<uint32_t>(k));
#pragma unroll
        for (int u = 0; u < U; ++u) q[k][u] = __uint_as_float(ld_shared_cluster_u32(peer + STEP * u * kSumLd * 4u));
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        v[u] = q[0][u];
#pragma unroll
        for (int k = 1; k < KS; ++k) v[u] += q[k][u];
      }
    }
    if (res) {
#pragma unroll
      for (int u = 0; u < U; ++u)
        if (lr + STEP * u < r1) add[u] = res[STEP * u * e.ld_residual];
      res += STEP * U * e.ld_residual;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (lr + STEP * u >= r1) break;
      const float pre = v[u] + bias;
      if (z) z[STEP * u * e.ld_z] = pre;
      const float out = activate(pre, e.act);
      y[STEP * u * e.ld_y] = res ? out + add[u] : out;
    }
    y += STEP * U * e.ld_y;
    if (z) z += STEP * U * e.ld_z;
  }
}

// The same for a tile with sums that are not finite or near the end of the accumulators' range, by ks
// ranks: such a sum is formed again from plain fp32 products of the operands, where an infinity meets no
// zeros among the other operand's parts and a large value is not rounded to one; the other sums stay as
// they are.  A sum that has become NaN is not looked at further.  16384 x 1024 -> 1024 takes 396 us, with one
// NaN 400 us, of NaN alone 8.3 ms, with every sum beyond 2^91 78 ms.
template <bool A_K, bool B_K>
__device__ __noinline__ void store_column_plain(const EpilogueF32& e, const float* a, int64_t lda, const float* b, int64_t ldb, int64_t K,
                                                int64_t row, int64_t row_end, int64_t col, const float* sum, int ks) {
  constexpr int STEP = kConvert / TN;
  const float* pb = B_K ? b + col * ldb : b + col;
  for (; row < row_end; row += STEP, sum += STEP * kSumLd) {
    const uint32_t at = smem_u32(sum);
    bool fine = true;
    float v = 0.0f;
    for (int k = 0; k < ks; ++k) {
      const float q = ks == 1 ? *sum : __uint_as_float(ld_shared_cluster_u32(mapa_shared(at, static_cast<uint32_t>(k))));
      fine = fine && fabsf(q) <= kLargest * kUnscale;
      v = k == 0 ? q : v + q;
    }
    if (!fine) {
      const float* pa = A_K ? a + row * lda : a + row;
      v = 0.0f;
      for (int64_t k0 = 0; k0 < K && v == v; k0 += 128) {
        float part = 0.0f;
        for (int64_t k = k0; k < min(K, k0 + 128); ++k) part = fmaf(pa[A_K ? k : k * lda], pb[B_K ? k : k * ldb], part);
        v += part;
      }
    }
    if (e.bias) v += e.bias[col];
    if (e.z) e.z[row * e.ld_z + col] = v;
    v = activate(v, e.act);
    if (e.residual) v += e.residual[row * e.ld_residual + col];
    e.y[row * e.ld_y + col] = v;
  }
}

__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err, uint32_t code) {
  return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, err, code));
}

// One tile of a product, by a cluster of ks CTAs.
template <bool A_K, bool B_K>
__device__ __forceinline__ void compute_tile(const ProductF32& job, int64_t m_tile, int64_t n_tile, const ColumnSums& cs, uint32_t* err,
                                             const int ks) {
  const float *const a = job.a, *const b = job.b;
  const int64_t lda = job.lda, ldb = job.ldb, M = job.M, N = job.N, K = job.K;
  const EpilogueF32 e = job.e;  // a copy: its address, which store_column_plain takes, keeps registers free in the loop
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);
  uint64_t* empty = full + kStages;
  uint64_t* cfull = empty + kStages;   // an accumulator holds its products
  uint64_t* cempty = cfull + 2;        // it has been added up
  uint64_t* mma_done = cempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);
  volatile int* wild = abort_flag + 1;  // a sum that is not finite, or large
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], kConvert / 32);
      mbar_init(&empty[s], 1);
    }
    for (int c = 0; c < 2; ++c) {
      mbar_init(&cfull[c], 1);
      mbar_init(&cempty[c], kConvert / 32);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    *wild = 0;
    fence_mbar_init();
  }
  if (warp == kConvert / 32) {
    tmem_alloc(tmem_holder, 512);
    tmem_relinquish();
  }
  tc_fence_before_sync();
  __syncthreads();
  tc_fence_after_sync();
  const uint32_t tmem = *tmem_holder;
  if (threadIdx.x == 0) launch_dependents();
  grid_dependency_wait();

  const int rank = ks > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int64_t m0 = m_tile * TM, n0 = n_tile * TN;
  const int64_t all_stages = (K + TK - 1) / TK, first = all_stages * rank / ks;
  const int stages = static_cast<int>(all_stages * (rank + 1) / ks - first);  // this rank's
  float* sums = reinterpret_cast<float*>(smem);  // [TM][kSumLd], once the ring is done with
  if (!A_K && cs.out && n_tile == 0 && rank == 0 && threadIdx.x < TM && m0 + threadIdx.x < M) {
    // the bias gradient of dW's rows, from the strips' sums in order
    float sum = 0.0f;
#pragma unroll 8
    for (int i = 0; i < cs.strips; ++i) sum += cs.sums[i * M + m0 + threadIdx.x];
    cs.out[m0 + threadIdx.x] = sum;
  }
  if (warp < kConvert / 32) {
    // ------------------------------------------------------------------ load and split, add up
    Share<TM, A_K> pa(a, lda, m0, M, first * TK);
    Share<TN, B_K> pb(b, ldb, n0, N, first * TK);
    int left = static_cast<int>(min(K - first * TK, int64_t(1) << 30));  // contraction indices from the next stage on
    auto load_all = [&] {
#pragma unroll
      for (int j = 0; j < pa.PIECES; ++j) pa.load(j, left);
#pragma unroll
      for (int j = 0; j < pb.PIECES; ++j) pb.load(j, left);
    };
    load_all();
    // Rows 32 (warp % 4) + lane, columns 16 (warp / 4) ..
    const int quad = warp & 3, col = (warp >> 2) * 16;
    float v[16];
#pragma unroll
    for (int j = 0; j < 16; ++j) v[j] = 0.0f;
    const int chunks = (stages + kFlush - 1) / kFlush;
    int chunk = 0;  // the next one to add up
    bool ok = true;
    auto add_up = [&] {
      const int c = chunk & 1;
      ok = ok && warp_wait(&cfull[c], static_cast<uint32_t>(chunk >> 1 & 1), abort_flag, err, kErrTimeoutEpilogue);
      ++chunk;
      if (!ok) return;
      tc_fence_after_sync();
      const uint32_t from = tmem + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(c * kAccCols + col);
      uint32_t big[16], mid[16], low[16];
      tmem_ld16(from, big);
      tmem_ld16(from + TN, mid);
      tmem_ld16(from + 2 * TN, low);
      asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        asm volatile("" : "+r"(big[j]), "+r"(mid[j]), "+r"(low[j]));
        v[j] += __uint_as_float(big[j]) + (__uint_as_float(mid[j]) + __uint_as_float(low[j]));
      }
      tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) mbar_arrive(&cempty[c]);
    };
    int stage = 0;
    uint32_t phase = 0;
    for (int s = 0; s < stages && ok; ++s) {
      // the accumulator before the present one, once its last MMAs have had a stage's time
      if (s % kFlush == 1 && s > kFlush) add_up();
      ok = ok && warp_wait(&empty[stage], phase ^ 1, abort_flag, err, kErrTimeoutProducer);
      if (!ok) break;
      uint8_t* to = smem + stage * kStageBytes;
      // a piece's next loads start as soon as it is split
      left -= TK;
      pa.advance();
      pb.advance();
#pragma unroll
      for (int j = 0; j < pa.PIECES; ++j) {
        pa.store(j, to);
        pa.load(j, left);
      }
#pragma unroll
      for (int j = 0; j < pb.PIECES; ++j) {
        pb.store(j, to + 3 * kABytes);
        pb.load(j, left);
      }
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive(&full[stage]);
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    while (ok && chunk < chunks) add_up();
    // The last accumulator is complete, so every MMA has read the ring.
    if (ok) {
      bool fine = true;
#pragma unroll
      for (int j = 0; j < 16; ++j) {
        sums[(quad * 32 + lane) * kSumLd + col + j] = v[j] * kUnscale;
        fine = fine && fabsf(v[j]) <= kLargest;
      }
      if (!fine && m0 + quad * 32 + lane < M) *wild = 1;
    }
  } else {
    // ------------------------------------------------------------------ MMAs
    const uint32_t ring = smem_u32(smem);
    int stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    for (int s = 0; s < stages; ++s) {
      const int chunk = s / kFlush, c = chunk & 1;
      if (s % kFlush == 0) ok = ok && warp_wait(&cempty[c], static_cast<uint32_t>(chunk >> 1 & 1) ^ 1u, abort_flag, err, kErrTimeoutMma);
      ok = ok && warp_wait(&full[stage], phase, abort_flag, err, kErrTimeoutMma);
      tc_fence_after_sync();
      if (lane == 0 && ok) {
        const uint32_t at = ring + static_cast<uint32_t>(stage) * kStageBytes, d = tmem + static_cast<uint32_t>(c * kAccCols);
        const uint64_t b0 = sdesc_sw128(at + 3 * kABytes, 16, 1024);
        const uint64_t a0 = sdesc_sw128(at, 16, 1024), a1 = sdesc_sw128(at + kABytes, 16, 1024), a2 = sdesc_sw128(at + 2 * kABytes, 16, 1024);
#pragma unroll
        for (int k = 0; k < TK / 16; ++k) {
          const uint32_t more = s % kFlush != 0 || k > 0 ? 1u : 0u;
          umma_bf16(d, a0 + 2 * k, b0 + 2 * k, idesc_bf16(TM, 3 * TN, false), more);
          umma_bf16(d + TN, a1 + 2 * k, b0 + 2 * k, idesc_bf16(TM, 2 * TN, false), 1u);
          umma_bf16(d + TN, a2 + 2 * k, b0 + 2 * k, idesc_bf16(TM, TN, false), 1u);
        }
        umma_commit(&empty[stage]);
        if (s % kFlush == kFlush - 1 || s + 1 == stages) umma_commit(&cfull[c]);
      }
      __syncwarp();
      if (++stage == kStages) {
        stage = 0;
        phase ^= 1;
      }
    }
    if (lane == 0) {  // every MMA issued completes before TMEM and the ring are given up
      umma_commit(mma_done);
      volatile int never = 0;
      mbar_wait(mma_done, 0, &never, err, kErrTimeoutMma);
    }
    __syncwarp();
  }
  tc_fence_before_sync();
  __syncthreads();
  if (warp == kConvert / 32) {
    tc_fence_after_sync();
    tmem_dealloc(tmem, 512);
  }
  if (ks > 1) cluster_sync();  // every rank's sums are in place
  // A thread stores one column of every eighth row.
  const int rows = static_cast<int>(min(int64_t(TM), M - m0)), r1 = rows * (rank + 1) / ks;
  const int lc = static_cast<int>(threadIdx.x) % TN, lr = rows * rank / ks + static_cast<int>(threadIdx.x) / TN;
  const int64_t row = m0 + lr, col = n0 + lc;
  bool large = *wild;
  for (int k = 0; k < ks && ks > 1; ++k)
    large |= ld_shared_cluster_u32(mapa_shared(smem_u32(const_cast<int*>(wild)), static_cast<uint32_t>(k))) != 0;
  if (threadIdx.x < kConvert && col < N) {
    const float bias = e.bias ? e.bias[col] : 0.0f;
    const float* sum = sums + lr * kSumLd + lc;
    float* y = e.y + row * e.ld_y + col;
    const float* res = e.residual ? e.residual + row * e.ld_residual + col : nullptr;
    float* z = e.z ? e.z + row * e.ld_z + col : nullptr;
    if (large) store_column_plain<A_K, B_K>(e, a, lda, b, ldb, K, row, m0 + r1, col, sum, ks);
    else if (ks == 1) store_column<1>(e, lr, r1, sum, bias, y, res, z);
    else if (ks == 2) store_column<2>(e, lr, r1, sum, bias, y, res, z);
    else if (ks == 4) store_column<4>(e, lr, r1, sum, bias, y, res, z);
    else store_column<8>(e, lr, r1, sum, bias, y, res, z);
  }
  if (ks > 1) {
    __syncwarp();
    cluster_sync();  // no CTA leaves while another still reads its sums
  }
}

template <bool A_K, bool B_K>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_f32(const __grid_constant__ ProductF32 job, const ColumnSums cs, uint32_t* err, const int ks) {
  compute_tile<A_K, B_K>(job, blockIdx.x / ks, blockIdx.y, cs, err, ks);
}

// The tiles of dx, then those of dW: for small layers, whose tiles leave SMs idle in two launches and
// whose launches are mostly start and end (128 rows, 256 -> 640: 11.3 us, where two launches took 19.8).
// A rank may have no stage of the shorter contraction; its sums are then zeros.
__global__ void __launch_bounds__(kThreads, 1)
    k_linear_f32_grads(const __grid_constant__ ProductF32 dx, const __grid_constant__ ProductF32 dw, const int dx_tiles, const ColumnSums cs,
                       uint32_t* err, const int ks) {
  const int t = static_cast<int>(blockIdx.x) / ks;
  if (t < dx_tiles) {
    const int n = static_cast<int>((dx.N + TN - 1) / TN);
    compute_tile<true, false>(dx, t / n, t % n, cs, err, ks);
  } else {
    const int n = static_cast<int>((dw.N + TN - 1) / TN);
    compute_tile<false, false>(dw, (t - dx_tiles) / n, (t - dx_tiles) % n, cs, err, ks);
  }
}

int64_t tiles_of(const ProductF32& p) { return (p.M + TM - 1) / TM * ((p.N + TN - 1) / TN); }
int64_t stages_of(const ProductF32& p) { return (p.K + TK - 1) / TK; }

// The split that leaves no SM a second CTA (15 clusters of eight and 33 of four fit 148 SMs), two
// stages a rank at least (of the longer contraction, where two products share a launch).
int split_of(int64_t tiles, int64_t stages, int sms) {
  return tiles <= sms * 15 / 148 && stages >= 16 ? 8
         : tiles <= sms * 33 / 148 && stages >= 8 ? 4
         : tiles * 2 <= sms && stages >= 4        ? 2
                                                  : 1;
}

template <auto KERNEL, typename... Params>
cudaError_t launch(dim3 grid, int ks, cudaStream_t s, const Params&... params) {
  static thread_local uint64_t ready = 0;  // devices on which the shared-memory limit is raised
  int dev = 0;
  if (cudaError_t r = cudaGetDevice(&dev)) return r;
  if (dev >= 64 || !(ready >> dev & 1u)) {
    if (cudaError_t r = cudaFuncSetAttribute(KERNEL, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem)) return r;
    if (dev < 64) ready |= uint64_t(1) << dev;
  }
  if (ks == 1) return launch_pdl(KERNEL, grid, dim3(kThreads), kSmem, s, params...);
  return launch_pdl_cluster(KERNEL, grid, dim3(kThreads), kSmem, s, static_cast<unsigned>(ks), params...);
}

template <bool A_K, bool B_K>
cudaError_t launch_product(const ProductF32& p, const ColumnSums& cs, uint32_t* err, int sms, cudaStream_t s) {
  const int ks = split_of(tiles_of(p), stages_of(p), sms);
  const dim3 grid(static_cast<unsigned>((p.M + TM - 1) / TM * ks), static_cast<unsigned>((p.N + TN - 1) / TN));
  return launch<k_linear_f32<A_K, B_K>>(grid, ks, s, p, cs, err, ks);
}

// ---------------------------------------------------------------------------- a few rows
// y of one to four rows: a warp streams the weights of an output feature at a time against the rows
// of x in shared memory, as k_linear_few does for bf16 (1 x 1024 x 1024: 3.1 us, where a 128-row tile
// takes 12 us; 1 x 4608 x 4608: 23.8 us, 12.9 of them its 85 MB at the copy rate: the stream starts only once
// x is staged).
constexpr int kFewThreads = 256, kFewSmem = 48 * 1024;

template <int R>
__global__ void __launch_bounds__(kFewThreads) k_linear_few_f32(const float* x, int64_t ld_x, const float* w, int64_t ld_w, int rows,
                                                                int N, int K, bool vec, const EpilogueF32 e) {
  extern __shared__ float sx[];  // [R][K rounded up to 4]
  const int lane = threadIdx.x & 31, ld_s = (K + 3) / 4 * 4;
  launch_dependents();
  grid_dependency_wait();
  for (int i = threadIdx.x; i < R * ld_s; i += kFewThreads) {
    const int r = i / ld_s, k = i - r * ld_s;
    sx[i] = r < rows && k < K ? x[r * ld_x + k] : 0.0f;
  }
  __syncthreads();
  const int warps = static_cast<int>(gridDim.x) * (kFewThreads / 32);
  for (int f = static_cast<int>(blockIdx.x) * (kFewThreads / 32) + (threadIdx.x >> 5); f < N; f += warps) {
    const float* wf = w + static_cast<int64_t>(f) * ld_w;
    float acc[R] = {};
    int k = 0;
    if (vec) {
#pragma unroll 4
      for (; k + 128 <= K; k += 128) {
        const float4 q = *reinterpret_cast<const float4*>(wf + k + 4 * lane);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const float4 v = *reinterpret_cast<const float4*>(sx + r * ld_s + k + 4 * lane);
          acc[r] = fmaf(q.x, v.x, fmaf(q.y, v.y, fmaf(q.z, v.z, fmaf(q.w, v.w, acc[r]))));
        }
      }
    }
#pragma unroll 4
    for (int i = k + lane; i < K; i += 32) {
      const float q = wf[i];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = fmaf(q, sx[r * ld_s + i], acc[r]);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] += __shfl_xor_sync(0xffffffffu, acc[r], o);
    float v = acc[0];
#pragma unroll
    for (int r = 1; r < R; ++r)
      if (lane == r) v = acc[r];
    if (lane < rows) {  // lane r finishes row r
      if (e.bias) v += e.bias[f];
      if (e.z) e.z[lane * e.ld_z + f] = v;
      if (e.act == DSV4V_ACT_GELU) v = 0.5f * v * (1.0f + erff(v * 0.70710678118654752f));
      else if (e.act == DSV4V_ACT_SILU) v = v / (1.0f + expf(-v));
      if (e.residual) v += e.residual[lane * e.ld_residual + f];
      e.y[lane * e.ld_y + f] = v;
    }
  }
}

template <int R>
cudaError_t launch_few(const ProductF32& p, int sms, cudaStream_t s) {
  const int64_t per = kFewThreads / 32;
  const int grid = static_cast<int>(std::min<int64_t>((p.N + per - 1) / per, sms * 4));
  const bool vec = (reinterpret_cast<uintptr_t>(p.b) & 15) == 0 && p.ldb % 4 == 0;
  return launch_pdl(k_linear_few_f32<R>, dim3(grid), dim3(kFewThreads), static_cast<size_t>(R) * ((p.K + 3) / 4 * 16), s, p.a, p.lda, p.b,
                    p.ldb, static_cast<int>(p.M), static_cast<int>(p.N), static_cast<int>(p.K), vec, p.e);
}

}  // namespace

cudaError_t launch_linear_f32(LinearForm form, const ProductF32& p, const ColumnSums& cs, uint32_t* err, int sms, cudaStream_t s) {
  if (form == LINEAR_FORWARD && p.M <= 4 && (p.M <= 2 ? p.M : 4) * ((p.K + 3) / 4 * 16) <= kFewSmem)
    return p.M == 1   ? launch_few<1>(p, sms, s)
           : p.M == 2 ? launch_few<2>(p, sms, s)
                      : launch_few<4>(p, sms, s);
  switch (form) {
    case LINEAR_FORWARD: return launch_product<true, true>(p, cs, err, sms, s);
    case LINEAR_INPUT_GRAD: return launch_product<true, false>(p, cs, err, sms, s);
    case LINEAR_WEIGHT_GRAD: return launch_product<false, false>(p, cs, err, sms, s);
    default: return cudaErrorInvalidValue;
  }
}

cudaError_t launch_linear_f32_grads(const ProductF32& dx, const ProductF32& dw, const ColumnSums& cs, uint32_t* err, int sms,
                                    cudaStream_t s) {
  const int64_t tiles = tiles_of(dx) + tiles_of(dw);
  if (tiles > sms) {
    if (cudaError_t r = launch_product<true, false>(dx, ColumnSums(), err, sms, s)) return r;
    return launch_product<false, false>(dw, cs, err, sms, s);
  }
  const int ks = split_of(tiles, std::max(stages_of(dx), stages_of(dw)), sms);
  return launch<k_linear_f32_grads>(dim3(static_cast<unsigned>(tiles * ks)), ks, s, dx, dw, static_cast<int>(tiles_of(dx)), cs, err, ks);
}

}  // namespace dsv4v
