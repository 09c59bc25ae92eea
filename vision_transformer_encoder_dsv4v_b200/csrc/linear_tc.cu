// The Linear layer on tcgen05: y = act(x W^T + b) + r and, for its backward, dx = dz W and
// dW = dz^T x.  One GEMM kernel D[M, N] = A . B^T serves the three, the two gradients also side by
// side in one launch; what differs is how the operands lie in memory (K-major: rows of the
// contraction; MN-major: columns) and the epilogue.
//
// Against the block's GEMM (gemm_tc.cu) this one takes any extent: TMA fills what lies outside the
// tensors with zeros, and the epilogue stores row segments through shared memory, so that rows,
// columns and row strides need not divide into tiles, boxes or vectors.
//
// Bounds and tiles.  What an SM takes in limits the main loop before the tensor pipe does: TMA
// brings about 65 bytes a clock into an SM, and a 128 x N x 64 step needs (128 + N) 128 bytes for
// 2 N clocks of MMA: 750 against 512 clocks at N = 256.  A pair of CTAs (cta_group::2) shares one B
// tile, which balances the two.  So large products run on pairs; single CTAs serve small ones,
// split along K over a cluster where there are fewer tiles than SMs.  Each split writes its fp32
// partial to its own shared memory and finishes a share of the tile, reading the partials of the
// others through distributed shared memory in rank order: no workspace, no atomics, one result.
//
// Roles (320 threads): warp 0 loads by TMA, warp 1 issues the MMAs, warps 2 to 9 finish tiles.  The
// accumulator is double-buffered in TMEM, so a tile's epilogue runs under the next tile's MMAs.
#include <algorithm>

#include "common.cuh"
#include "internal.h"
#include "linear.h"

namespace dsv4v {

namespace {

constexpr int BM = 128;
constexpr int BK = 64;
constexpr int kEpiWarps = 8;
constexpr int kThreads = 64 + 32 * kEpiWarps;
constexpr int kMaxDynSmem = 232448;        // 227 KB per CTA
constexpr int kBoxBytes = 2048, kBiasBytes = 512;  // per epilogue warp: 32 rows x 64 bytes, and the bias of 4 x 32 columns
constexpr int kStagingBytes = kEpiWarps * (kBoxBytes + kBiasBytes);
constexpr int kPartPad = 4;  // puts the rows of a warp's 16-byte accesses to a partial on different banks
constexpr int kGroupM = 8;                 // row tiles of a raster group

template <int BN, bool PAIR>
struct Tile {
  // A stage holds KPS 64-deep steps: a narrow tile's single step is shorter than the hand-over of a
  // stage (about 240 clocks) and too few bytes in flight to hide memory.
  static constexpr int KPS = BN <= 192 ? 2 : 1;
  static constexpr int B_ROWS = PAIR ? BN / 2 : BN;
  static constexpr int B_BYTES = B_ROWS * BK * 2;
  static constexpr int OFF_BARRIERS = (kMaxDynSmem - 1024 - 512 - kStagingBytes) & ~1023;
  static constexpr int OFF_STAGING = OFF_BARRIERS + 512;
  static constexpr int SMEM = 1024 + OFF_STAGING + kStagingBytes;
  static constexpr int RING = OFF_BARRIERS;
  static constexpr int TMEM_COLS = 2 * BN <= 128 ? 128 : (2 * BN <= 256 ? 256 : 512);  // two accumulators
  static constexpr int PART_LD = BN + kPartPad;  // row stride, in floats, of a split's fp32 partial in the ring
  static_assert(PAIR || BM * PART_LD * 4 <= RING, "a partial tile has to fit the ring");
};
constexpr int kMaxStages = 16;

// ---------------------------------------------------------------------------- barriers
// The load and MMA warps run their loops as whole warps, with one lane issuing: their counters and
// descriptors then live in uniform registers, which the issued instructions take their operands
// from.  As one lane's loops they cost 380 and 550 clocks a step, more than a narrow tile's work.
// Barriers go by their shared-memory address, and the waits are those of common.cuh.
template <bool CLUSTER>
__device__ __forceinline__ bool bar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  if constexpr (CLUSTER)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(bar), "r"(parity)
        : "memory");
  return ok != 0;
}
template <bool CLUSTER>
__device__ __noinline__ bool bar_wait_long(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err, uint32_t code) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (bar_try<CLUSTER>(bar, parity)) return true;
    if ((i & 255u) == 0) {
      if (*abort_flag) return false;
      const uint64_t now = global_timer_ns();
      if (t0 == 0) {
        t0 = now;
      } else if (now - t0 > kWaitLimitNs) {
        atomicCAS(err, 0u, code);
        *abort_flag = 1;
        return false;
      }
    }
  }
}
// Every lane waits for the phase of the given parity; false once the wait has given up (see
// mbar_wait).  The instructions that follow gather the warp again by their election.
template <bool CLUSTER = false>
__device__ __forceinline__ bool bar_wait(uint32_t bar, uint32_t parity, volatile int* abort_flag, uint32_t* err, uint32_t code) {
#pragma unroll 1
  for (int i = 0; i < 8; ++i)
    if (bar_try<CLUSTER>(bar, parity)) return true;
  return bar_wait_long<CLUSTER>(bar, parity, abort_flag, err, code);
}

// The instructions below are executed by a whole, converged warp and issued by one of its lanes
// (always the same one) if that lane's `ok` holds: both are part of the instruction's own predicate,
// not a branch, which lanes whose waits ended differently could take differently.
#define ELECTED(ok, body) "{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tsetp.ne.and.b32 q, " ok ", 0, q;\n\t" body "}"

__device__ __forceinline__ bool elected() {
  uint32_t r;
  asm volatile("{\n\t.reg .pred q;\n\telect.sync _|q, 0xffffffff;\n\tselp.u32 %0, 1, 0, q;\n\t}" : "=r"(r));
  return r != 0;
}

__device__ __forceinline__ void bar_expect(uint32_t bar, uint32_t bytes, uint32_t ok) {
  asm volatile(ELECTED("%2", "@q mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t") ::"r"(bar), "r"(bytes), "r"(ok) : "memory");
}

// Tiled load of one box at (x, y) into this CTA's shared memory, counted on the barrier at `bar`
// (PAIR: a shared::cluster address, the leader's).
template <bool PAIR>
__device__ __forceinline__ void tma_tile(uint32_t dst, const CUtensorMap* map, uint32_t bar, int x, int y, uint32_t ok) {
  if constexpr (PAIR)
    asm volatile(ELECTED("%5", "@q cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                               " [%0], [%1, {%3, %4}], [%2];\n\t") ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(ok)
                 : "memory");
  else
    asm volatile(ELECTED("%5", "@q cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
                               " [%0], [%1, {%3, %4}], [%2];\n\t") ::"r"(dst),
                 "l"(reinterpret_cast<uint64_t>(map)), "r"(bar), "r"(x), "r"(y), "r"(ok)
                 : "memory");
}

// D[tmem] (+)= A[smem] * B[smem]^T; PAIR: of both CTAs, M = 256.
template <bool PAIR>
__device__ __forceinline__ void mma_step(uint32_t d_tmem, uint64_t a_desc, uint64_t b_desc, uint32_t idesc, uint32_t accumulate,
                                         uint32_t ok) {
  if constexpr (PAIR)
    asm volatile(ELECTED("%5", ".reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                               "@q tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t") ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(ok)
                 : "memory");
  else
    asm volatile(ELECTED("%5", ".reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                               "@q tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t") ::"r"(d_tmem),
                 "l"(a_desc), "l"(b_desc), "r"(idesc), "r"(accumulate), "r"(ok)
                 : "memory");
}

// Arrives on the barrier (PAIR: on both CTAs') when every MMA issued so far has completed.
template <bool PAIR>
__device__ __forceinline__ void commit_to(uint32_t bar, uint32_t ok) {
  if constexpr (PAIR)
    asm volatile(ELECTED("%2", "@q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n\t") ::"r"(bar),
                 "h"(static_cast<uint16_t>(3)), "r"(ok)
                 : "memory");
  else
    asm volatile(ELECTED("%1", "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t") ::"r"(bar), "r"(ok) : "memory");
}

// One product of a launch.
struct Job {
  int M, N;              // extents of D
  int tiles_m, tiles_n;  // BM (PAIR: 2 BM) x BN tiles
  int kb_total;          // stages of the contraction, 64 KPS deep
  LinearEpilogue e;
};

struct Params {
  Job job[2];    // both gradients in one launch: the input's, the weight's
  int units;     // CTAs (PAIR: pairs) that take the first of two jobs
  int a_rows;    // rows of a K-major A's boxes: fewer than BM where D has fewer (the MMA then reads
                 // what lies behind them, into accumulator rows that nobody looks at)
  int stages;    // of the ring
  ColumnSums cs; // weight gradient: the bias gradient that goes with it
  uint32_t* err;
};

// Tile t in an order that keeps the tiles in flight together compact (kGroupM row tiles by as many
// column tiles as it takes), so that they share their operands in L2: with whole columns of 64 row
// tiles a wave of the 16384 x 4096 x 4608 product would fetch 155 MB, with groups 40 MB.
__device__ __forceinline__ void tile_at(const Job& p, int t, int& m, int& n) {
  const int per = kGroupM * p.tiles_n, g = t / per, r = t - g * per;
  const int rows = min(kGroupM, p.tiles_m - g * kGroupM);
  n = r / rows;
  m = g * kGroupM + (r - n * rows);
}

// ---------------------------------------------------------------------------- epilogue math
// Both activations take 2^x and 1/x from the MUFU pipe (a few 2^-23 relative): two such operations
// an element keep a tile's epilogue under its main loop, which erff and expf would not (about 30
// instructions an element: 10,000 clocks a 128 x 256 tile).
//
// erf by Abramowitz and Stegun 7.1.26, |error| <= 1.5e-7: erfc(x) = poly(t) e^(-x^2), x >= 0.  Two
// values at a time, in packed fp32 instructions, which halves the issue slots that bound it (784 x
// 1024 x 2816, GELU: 13.5 -> 13.1 us).
__device__ __forceinline__ uint64_t both(float v) { return pk2(v, v); }
__device__ __forceinline__ void gelu_fast(float& a, float& b) {
  const uint64_t x = mul2(pk2(fabsf(a), fabsf(b)), both(0.70710678118654752f));
  const uint64_t e = mul2(mul2(x, x), both(-1.4426950408889634f));
  float t0, t1, e0, e1;
  upk2(fma2(both(0.3275911f), x, both(1.0f)), t0, t1);
  upk2(e, e0, e1);
  const uint64_t t = pk2(rcp_approx(t0), rcp_approx(t1));
  uint64_t q = fma2(both(1.061405429f * 0.5f), t, both(-1.453152027f * 0.5f));
  q = fma2(q, t, both(1.421413741f * 0.5f));
  q = fma2(q, t, both(-0.284496736f * 0.5f));
  q = fma2(q, t, both(0.254829592f * 0.5f));
  const uint64_t tail = mul2(mul2(q, t), pk2(ex2_approx(e0), ex2_approx(e1)));  // (1 - erf) / 2 at |x|
  float l0, l1, h0, h1;
  upk2(tail, l0, l1);
  upk2(sub2(both(1.0f), tail), h0, h1);
  upk2(mul2(pk2(a, b), pk2(a >= 0.0f ? h0 : l0, b >= 0.0f ? h1 : l1)), a, b);
}
__device__ __forceinline__ void silu_fast(float& a, float& b) {
  float e0, e1, d0, d1;
  const uint64_t z = pk2(a, b);
  upk2(mul2(z, both(-1.4426950408889634f)), e0, e1);
  upk2(add2(both(1.0f), pk2(ex2_approx(e0), ex2_approx(e1))), d0, d1);
  upk2(mul2(z, pk2(rcp_approx(d0), rcp_approx(d1))), a, b);
}
// An even number of values.
template <int N>
__device__ __forceinline__ void activate(float (&v)[N], int act) {
  if (act == DSV4V_ACT_GELU) {
#pragma unroll
    for (int j = 0; j < N; j += 2) gelu_fast(v[j], v[j + 1]);
  } else if (act == DSV4V_ACT_SILU) {
#pragma unroll
    for (int j = 0; j < N; j += 2) silu_fast(v[j], v[j + 1]);
  }
}

// 16-byte chunk `c` (0..3) of row `r` of a staging box: 32 rows of 64 bytes.  Eight lanes that
// take one chunk of eight rows, or the chunks of two rows, meet eight different 16-byte banks.
__device__ __forceinline__ uint4* box_at(uint8_t* box, int r, int c) {
  return reinterpret_cast<uint4*>(box + r * 64 + ((c ^ ((r >> 1) & 3)) << 4));
}

// Rows [row0, row0 + 32) x columns [col0, col0 + 32) of a bf16 matrix, between global memory and
// a staging box: lane l takes chunk l % 4 of rows l / 4 + 8 i.  `vec`: rows are 16-byte aligned.
__device__ __forceinline__ void fetch_box(const __nv_bfloat16* src, int64_t ld, int row0, int col0, int M, int N, bool vec,
                                          int lane, uint4 (&q)[4]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int r = row0 + (lane >> 2) + 8 * i, c = col0 + (lane & 3) * 8;
    q[i] = make_uint4(0, 0, 0, 0);
    if (r >= M || c >= N) continue;
    const __nv_bfloat16* p = src + static_cast<int64_t>(r) * ld + c;
    if (vec && c + 8 <= N) {
      q[i] = *reinterpret_cast<const uint4*>(p);
    } else {
      const uint16_t* u = reinterpret_cast<const uint16_t*>(p);
      uint32_t w[4] = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (c + j < N) w[j >> 1] |= static_cast<uint32_t>(u[j]) << (16 * (j & 1));
      q[i] = make_uint4(w[0], w[1], w[2], w[3]);
    }
  }
}

// Rows that are not 16-byte aligned leave through 2-byte stores, a row's 32 columns by the 32
// lanes, so that a store still covers whole sectors.
__device__ __forceinline__ void store_box(__nv_bfloat16* dst, int64_t ld, int row0, int col0, int M, int N, bool vec, int lane,
                                          uint8_t* box) {
  if (vec) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int lr = (lane >> 2) + 8 * i, r = row0 + lr, c = col0 + (lane & 3) * 8;
      if (r >= M || c >= N) continue;
      const uint4 q = *box_at(box, lr, lane & 3);
      __nv_bfloat16* p = dst + static_cast<int64_t>(r) * ld + c;
      if (c + 8 <= N) {
        *reinterpret_cast<uint4*>(p) = q;
      } else {
        const uint32_t w[4] = {q.x, q.y, q.z, q.w};
        uint16_t* u = reinterpret_cast<uint16_t*>(p);
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (c + j < N) u[j] = static_cast<uint16_t>(w[j >> 1] >> (16 * (j & 1)));
      }
    }
  } else if (col0 + lane < N) {
    const int rows = min(32, M - row0);
    for (int lr = 0; lr < rows; ++lr) {
      const uint16_t* u = reinterpret_cast<const uint16_t*>(box_at(box, lr, lane >> 3)) + (lane & 7);
      reinterpret_cast<uint16_t*>(dst + static_cast<int64_t>(row0 + lr) * ld + col0)[lane] = *u;
    }
  }
}

__device__ __forceinline__ uint4 pack8(const float* v) {
  return make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}

// The bias gradient of rows m0 .. m0 + 127 of dW: the strips' sums, in order.  The epilogue warps have
// the time of a tile's main loop for it.
__device__ __forceinline__ void sum_columns(const ColumnSums& cs, int M, int m0) {
  const int t = static_cast<int>(threadIdx.x) - 64, f = m0 + t;
  if (t >= BM || f >= M) return;
  float sum = 0.0f;
#pragma unroll 8
  for (int i = 0; i < cs.strips; ++i) sum += cs.sums[static_cast<int64_t>(i) * M + f];
  cs.out[f] = sum;
}

// Cluster split-K: this rank's share of a tile of `rows` rows from row m0 and COLS columns from column
// n0 of N.  The tile's 8-column pieces are dealt to the ranks in turn; a piece's partials are all
// fetched, then summed in rank order.
template <int COLS, bool FWD, int KS>
__device__ __forceinline__ void finish_pieces(const LinearEpilogue& e, float* part, int slice, int rows, int m0, int n0, int N) {
  constexpr int PIECES = COLS / 8, LD = COLS + kPartPad;
  uint32_t base[KS];
#pragma unroll
  for (int k = 0; k < KS; ++k) base[k] = mapa_shared(smem_u32(part), static_cast<uint32_t>(k));
  for (int i = (static_cast<int>(threadIdx.x) - 64) * KS + slice; i < rows * PIECES; i += 32 * kEpiWarps * KS) {
    const int lr = i / PIECES, c = (i - lr * PIECES) * 8;
    const int row = m0 + lr, col = n0 + c;
    if (col >= N) continue;
    const uint32_t at = static_cast<uint32_t>(lr * LD + c) * 4u;
    float4 q[KS][2];
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      q[k][0] = ld_shared_cluster_f4(base[k] + at);
      q[k][1] = ld_shared_cluster_f4(base[k] + at + 16);
    }
    float v[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
    for (int k = 0; k < KS; ++k) {
      v[0] += q[k][0].x, v[1] += q[k][0].y, v[2] += q[k][0].z, v[3] += q[k][0].w;
      v[4] += q[k][1].x, v[5] += q[k][1].y, v[6] += q[k][1].z, v[7] += q[k][1].w;
    }
    const int n = min(8, N - col);
    const bool whole = e.vec_io && n == 8;
    auto put = [&](__nv_bfloat16* dst) {
      if (whole) {
        *reinterpret_cast<uint4*>(dst) = pack8(v);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) dst[j] = __float2bfloat16_rn(v[j]);
      }
    };
    if constexpr (FWD) {
      if (e.bias) {
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (j < n) v[j] += e.bias[col + j];
      }
      if (e.z) put(e.z + static_cast<int64_t>(row) * e.ld_z + col);
      activate(v, e.act);
      if (e.residual) {
        const __nv_bfloat16* r = e.residual + static_cast<int64_t>(row) * e.ld_residual + col;
        if (whole) {
          const uint4 w4 = *reinterpret_cast<const uint4*>(r);
          const uint32_t w[4] = {w4.x, w4.y, w4.z, w4.w};
#pragma unroll
          for (int j = 0; j < 4; ++j) v[2 * j] += bf16_lo(w[j]), v[2 * j + 1] += bf16_hi(w[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 8; ++j)
            if (j < n) v[j] += __bfloat162float(r[j]);
        }
      }
    }
    put(e.y + static_cast<int64_t>(row) * e.ld_y + col);
  }
}

// The epilogue's warps meet.
__device__ __forceinline__ void epilogue_sync() { asm volatile("bar.sync 1, %0;" ::"n"(32 * kEpiWarps) : "memory"); }

// ---------------------------------------------------------------------------- kernel
// An MN-major operand is loaded as boxes of 64 columns of its stored [K, MN] matrix (atom columns of
// 64 KPS rows); else K-major, in boxes of 64 columns of its rows.  The forward has bias, activation,
// residual and the saved pre-activation; the gradients store D as it is.  LINEAR_BOTH_GRADS splits
// the CTAs between the two gradients.  LINEAR_FORWARD_SWAPPED forms D^T = W . x^T for few rows of x, one
// tile a cluster.  KS (cluster split-K) is the cluster's size, 1 to 8.
template <int BN, bool PAIR, LinearForm FORM>
__global__ void __launch_bounds__(kThreads, 1)
    k_linear(const __grid_constant__ CUtensorMap tm_a0, const __grid_constant__ CUtensorMap tm_b0,
             const __grid_constant__ CUtensorMap tm_a1, const __grid_constant__ CUtensorMap tm_b1,
             const __grid_constant__ Params p, const int ks) {
  constexpr bool BOTH = FORM == LINEAR_BOTH_GRADS, SWAP = FORM == LINEAR_FORWARD_SWAPPED, FWD = FORM == LINEAR_FORWARD || SWAP,
                 B_MN = !FWD;
  using T = Tile<BN, PAIR>;
  constexpr int KPS = T::KPS;
  constexpr int BMT = PAIR ? 2 * BM : BM;
  const int span = PAIR ? 2 : ks;  // CTAs that share a tile
  const int unit = static_cast<int>(blockIdx.x) / span, units = static_cast<int>(gridDim.x) / span;
  const bool second = BOTH && unit >= p.units;
  const Job& job = p.job[second ? 1 : 0];
  const bool a_mn = BOTH ? second : FORM == LINEAR_WEIGHT_GRAD;
  const CUtensorMap* tm_a = second ? &tm_a1 : &tm_a0;
  const CUtensorMap* tm_b = second ? &tm_b1 : &tm_b0;
  // One step's A and B; a stage is KPS A's, then KPS B's.  An MN-major operand's atom columns hold
  // the stage's whole depth.
  const uint32_t a_bytes = FORM == LINEAR_WEIGHT_GRAD ? BM * BK * 2 : static_cast<uint32_t>(p.a_rows) * BK * 2;
  const uint32_t stage_bytes = KPS * (a_bytes + T::B_BYTES);
  constexpr uint32_t kAtom = 8192 * KPS;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + T::OFF_BARRIERS);
  uint64_t* empty = full + kMaxStages;
  uint64_t* tfull = empty + kMaxStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* mma_done = tempty + 2;
  uint32_t* tmem_holder = reinterpret_cast<uint32_t*>(mma_done + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_holder + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const uint32_t crank = (PAIR || ks > 1) ? cluster_ctarank() : 0u;
  const uint32_t rank = PAIR ? crank : 0u;  // 0: the pair's leader, which issues the MMAs
  // This CTA's share of the contraction, and the tiles it takes.
  const int slice = ks > 1 ? static_cast<int>(crank) : 0;
  const int kb0 = static_cast<int>(static_cast<int64_t>(slice) * job.kb_total / ks);
  const int kb1 = static_cast<int>(static_cast<int64_t>(slice + 1) * job.kb_total / ks);
  const int t_first = second ? unit - p.units : unit, t_step = BOTH ? (second ? units - p.units : p.units) : units;
  const int tiles = job.tiles_m * job.tiles_n;

  if (threadIdx.x == 0) {
    for (int s = 0; s < p.stages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], (PAIR ? 2 : 1) * kEpiWarps);
    }
    mbar_init(mma_done, 1);
    *abort_flag = 0;
    fence_mbar_init();
    tma_prefetch_desc(tm_a);
    tma_prefetch_desc(tm_b);
  }
  if (warp == 1) {
    if constexpr (PAIR) {
      tmem_alloc_pair(tmem_holder, T::TMEM_COLS);
      tmem_relinquish_pair();
    } else {
      tmem_alloc(tmem_holder, T::TMEM_COLS);
      tmem_relinquish();
    }
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // both CTAs' barriers exist before any remote use
  tc_fence_after_sync();
  const uint32_t tmem_base = *tmem_holder;
  if constexpr (PAIR) {
    // The leader's MMAs write the same TMEM columns in both CTAs.
    if (threadIdx.x == 0 &&
        ld_shared_cluster_u32(mapa_shared(smem_u32(const_cast<uint32_t*>(tmem_holder)), rank ^ 1u)) != tmem_base) {
      atomicCAS(p.err, 0u, static_cast<uint32_t>(kErrPairTmem));
      *abort_flag = 1;
    }
  }
  if (threadIdx.x == 0) launch_dependents();
  // Every role waits here, so that a bounded wait below never counts a predecessor's run.
  grid_dependency_wait();

  if (warp == 0) {
    // ------------------------------------------------------------------ loads
    int stage = 0;
    uint32_t phase = 0, issued = 0, issued_phase = 0;
    bool ok = true;
    // Both CTAs of a pair complete a stage on the leader's barrier, for which the leader posts the
    // bytes.
    const uint32_t full_bar = smem_u32(full), empty_bar = smem_u32(empty), ring = smem_u32(smem);
    const uint32_t full_leader = PAIR ? mapa_shared(full_bar, 0) : full_bar;
    const bool posts = !PAIR || rank == 0;
    const uint32_t tx = (PAIR ? 2 : 1) * stage_bytes;
    for (int t = t_first; t < tiles; t += t_step) {
      int mt, nt;
      tile_at(job, t, mt, nt);
      const int m0 = mt * BMT + static_cast<int>(rank) * BM;
      const int n0 = nt * BN + static_cast<int>(rank) * (BN / 2) * (PAIR ? 1 : 0);
      for (int kb = kb0; kb < kb1; ++kb) {
        ok = ok && bar_wait(empty_bar + 8u * stage, phase ^ 1, abort_flag, p.err, kErrTimeoutProducer);
        const uint32_t sa = ring + static_cast<uint32_t>(stage) * stage_bytes, sb = sa + KPS * a_bytes, bar = full_leader + 8u * stage;
        if (posts) bar_expect(full_bar + 8u * stage, tx, ok);
        const int k0 = kb * (KPS * BK);
        if (a_mn) {
#pragma unroll
          for (int j = 0; j < BM / 64; ++j) tma_tile<PAIR>(sa + j * kAtom, tm_a, bar, m0 + 64 * j, k0, ok);
        } else {
#pragma unroll
          for (int j = 0; j < KPS; ++j) tma_tile<PAIR>(sa + j * a_bytes, tm_a, bar, k0 + j * BK, m0, ok);
        }
        if constexpr (B_MN) {
#pragma unroll
          for (int j = 0; j < T::B_ROWS / 64; ++j) tma_tile<PAIR>(sb + j * kAtom, tm_b, bar, n0 + 64 * j, k0, ok);
        } else {
#pragma unroll
          for (int j = 0; j < KPS; ++j) tma_tile<PAIR>(sb + j * T::B_BYTES, tm_b, bar, k0 + j * BK, n0, ok);
        }
        if (ok) {
          issued |= 1u << stage;
          issued_phase = (issued_phase & ~(1u << stage)) | (phase << stage);
        }
        if (++stage == p.stages) {
          stage = 0;
          phase ^= 1;
        }
      }
    }
    // No copy is in flight when the CTA exits: the MMAs consumed every stage, unless a wait gave
    // up; then wait for each one here.  The second CTA of a pair has no full barrier of its own
    // and waits for the MMAs' release of the stages that it filled.
    if (elected()) {
      volatile int never = 0;
      for (int s = 0; s < p.stages; ++s) {
        if (!(issued & (1u << s))) continue;
        mbar_wait(posts ? &full[s] : &empty[s], (issued_phase >> s) & 1u, &never, p.err, kErrTimeoutProducer);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    // ------------------------------------------------------------------ MMAs
    if (PAIR && rank != 0) {
      volatile int never = 0;  // its TMEM is written until the leader's final commit
      mbar_wait(mma_done, 0, &never, p.err, kErrTimeoutMma);
    } else {
      const uint32_t idesc = a_mn ? idesc_bf16_mn(BMT, BN, true, B_MN) : idesc_bf16_mn(BMT, BN, false, B_MN);
      const uint32_t step_a = a_mn ? 128 : 2;  // 16 of K, in 16-byte units
      constexpr uint32_t kStepB = B_MN ? 128 : 2;
      const uint32_t full_bar = smem_u32(full), empty_bar = smem_u32(empty), tfull_bar = smem_u32(tfull), tempty_bar = smem_u32(tempty);
      const uint64_t adesc0 = sdesc_sw128(smem_u32(smem), a_mn ? kAtom : 16, 1024);
      const uint64_t bdesc0 = sdesc_sw128(smem_u32(smem) + KPS * a_bytes, B_MN ? kAtom : 16, 1024);
      int stage = 0, acc = 0;
      uint32_t phase = 0, acc_phase = 0;
      bool ok = true;
      for (int t = t_first; t < tiles; t += t_step) {
        ok = ok && bar_wait<PAIR>(tempty_bar + 8u * acc, acc_phase ^ 1, abort_flag, p.err, kErrTimeoutMma);
        tc_fence_after_sync();
        const uint32_t d_tmem = tmem_base + static_cast<uint32_t>(acc * BN);
        for (int kb = kb0; kb < kb1; ++kb) {
          ok = ok && bar_wait(full_bar + 8u * stage, phase, abort_flag, p.err, kErrTimeoutMma);
          tc_fence_after_sync();
          const uint32_t at = static_cast<uint32_t>(stage) * (stage_bytes / 16);
#pragma unroll
          for (int j = 0; j < KPS; ++j) {
            // a step deeper: the next tile of a K-major operand, 64 rows on in an MN-major one
            const uint64_t adesc = adesc0 + (at + (a_mn ? j * 512u : j * (a_bytes / 16)));
            const uint64_t bdesc = bdesc0 + (at + (B_MN ? j * 512u : j * (T::B_BYTES / 16u)));
#pragma unroll
            for (int k = 0; k < BK / 16; ++k) {
              const uint32_t accum = (kb > kb0 || j > 0 || k > 0) ? 1u : 0u;
              mma_step<PAIR>(d_tmem, adesc + step_a * k, bdesc + kStepB * k, idesc, accum, ok);
            }
          }
          commit_to<PAIR>(empty_bar + 8u * stage, ok);
          if (++stage == p.stages) {
            stage = 0;
            phase ^= 1;
          }
        }
        commit_to<PAIR>(tfull_bar + 8u * acc, ok);
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
      // Every MMA issued completes before TMEM is released.
      commit_to<PAIR>(smem_u32(mma_done), 1u);
      volatile int never = 0;
      mbar_wait(mma_done, 0, &never, p.err, kErrTimeoutMma);
    }
    __syncwarp();
    if (!PAIR && ks > 1) {
      cluster_sync();
      cluster_sync();
    }
  } else {
    // ------------------------------------------------------------------ epilogue
    const int quad = warp & 3;           // TMEM lanes [32 quad, 32 quad + 32) belong to this warp
    const int half = (warp - 2) >> 2;    // column groups half, half + 2, ...
    const LinearEpilogue& e = job.e;
    constexpr int NG = BN / 32;
    uint8_t* box = smem + T::OFF_STAGING + (warp - 2) * kBoxBytes;
    float* bias_s = reinterpret_cast<float*>(smem + T::OFF_STAGING + kEpiWarps * kBoxBytes + (warp - 2) * kBiasBytes);
    const uint32_t tempty_leader = PAIR ? mapa_shared(smem_u32(tempty), 0) : 0u;
    int acc = 0;
    uint32_t acc_phase = 0;
    if constexpr (SWAP) {
      // One tile of 128 features a cluster, whose partial is turned round on its way to the ring.
      constexpr int LD = BM + kPartPad;
      static_assert(!PAIR && BN * LD * 4 <= T::RING, "the partial has to fit the ring");
      const int f0 = t_first * BM, rows = job.N;
      const bool got = mbar_wait(&tfull[0], 0, abort_flag, p.err, kErrTimeoutEpilogue);
      const bool all_got = __all_sync(0xffffffffu, got);
      tc_fence_after_sync();
      float* part = reinterpret_cast<float*>(smem);
      if (all_got && f0 + quad * 32 < job.M) {
#pragma unroll 1
        for (int r0 = 16 * half; r0 < rows; r0 += 32) {
          uint32_t r[16];
          tmem_ld16(tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(r0), r);
          asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
          for (int j = 0; j < 16; ++j) {
            asm volatile("" : "+r"(r[j]));
            if (r0 + j < rows) part[(r0 + j) * LD + quad * 32 + lane] = __uint_as_float(r[j]);
          }
        }
      }
      __syncwarp();
      if (ks == 1) epilogue_sync();
      else cluster_sync();
      if (ks == 1) finish_pieces<BM, FWD, 1>(e, part, 0, rows, 0, f0, job.M);
      else finish_pieces<BM, FWD, 2>(e, part, slice, rows, 0, f0, job.M);
      __syncwarp();
      if (ks > 1) cluster_sync();  // no CTA leaves while another still reads its partial
    } else if (PAIR || ks == 1) {
      for (int t = t_first; t < tiles; t += t_step) {
        int mt, nt;
        tile_at(job, t, mt, nt);
        const int row0 = mt * BMT + static_cast<int>(rank) * BM + quad * 32;
        const int n0 = nt * BN;
        if (!FWD && a_mn && p.cs.out && nt == 0) sum_columns(p.cs, job.M, mt * BMT + static_cast<int>(rank) * BM);
        uint4 res[4];
        if (FWD && e.residual) fetch_box(e.residual, e.ld_residual, row0, n0 + 32 * half, job.M, job.N, e.vec_io, lane, res);
        if (FWD && e.bias) {  // this warp's columns, under the main loop
#pragma unroll
          for (int g = half; g < NG; g += 2) {
            const int c = n0 + 32 * g + lane;
            bias_s[16 * (g - half) + lane] = c < job.N ? e.bias[c] : 0.0f;
          }
          __syncwarp();
        }
        const bool got = mbar_wait(&tfull[acc], acc_phase, abort_flag, p.err, kErrTimeoutEpilogue);
        if (!__all_sync(0xffffffffu, got)) break;
        tc_fence_after_sync();
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quad * 32) << 16) + static_cast<uint32_t>(acc * BN);
#pragma unroll 1
        for (int g = half; g < NG; g += 2) {
          uint32_t r[32];
          tmem_ld32(t_row + g * 32, r);
          if (FWD && e.residual) {
#pragma unroll
            for (int i = 0; i < 4; ++i) *box_at(box, (lane >> 2) + 8 * i, lane & 3) = res[i];
            if (g + 2 < NG) fetch_box(e.residual, e.ld_residual, row0, n0 + 32 * (g + 2), job.M, job.N, e.vec_io, lane, res);
            __syncwarp();
          }
          float v[32];
          tmem_ld_wait(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          if (g + 2 >= NG) {  // this warp's last read of the accumulator
            tc_fence_before_sync();
            __syncwarp();
            if (lane == 0) {
              if constexpr (PAIR) mbar_arrive_cluster(tempty_leader + 8u * static_cast<uint32_t>(acc));
              else mbar_arrive(&tempty[acc]);
            }
          }
          const int col0 = n0 + 32 * g;
          if constexpr (FWD) {
            if (e.bias) {
#pragma unroll
              for (int q = 0; q < 8; ++q) {
                const float4 b = reinterpret_cast<const float4*>(bias_s + 16 * (g - half))[q];
                v[4 * q] += b.x, v[4 * q + 1] += b.y, v[4 * q + 2] += b.z, v[4 * q + 3] += b.w;
              }
            }
            uint4 own_res[4];
            if (e.residual) {
#pragma unroll
              for (int c = 0; c < 4; ++c) own_res[c] = *box_at(box, lane, c);
              __syncwarp();
            }
            if (e.z) {
#pragma unroll
              for (int c = 0; c < 4; ++c) *box_at(box, lane, c) = pack8(v + 8 * c);
              __syncwarp();
              store_box(e.z, e.ld_z, row0, col0, job.M, job.N, e.vec_io, lane, box);
              __syncwarp();
            }
            activate(v, e.act);
            if (e.residual) {
#pragma unroll
              for (int c = 0; c < 4; ++c) {
                const uint32_t w[4] = {own_res[c].x, own_res[c].y, own_res[c].z, own_res[c].w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                  v[8 * c + 2 * j] += bf16_lo(w[j]);
                  v[8 * c + 2 * j + 1] += bf16_hi(w[j]);
                }
              }
            }
          }
#pragma unroll
          for (int c = 0; c < 4; ++c) *box_at(box, lane, c) = pack8(v + 8 * c);
          __syncwarp();
          store_box(e.y, e.ld_y, row0, col0, job.M, job.N, e.vec_io, lane, box);
          __syncwarp();
        }
        if (++acc == 2) {
          acc = 0;
          acc_phase ^= 1;
        }
      }
    } else {
      // Cluster split-K: one tile a cluster.  The partial goes to the ring, which the MMAs are
      // done with; only rows that exist are kept.
      int mt, nt;
      tile_at(job, t_first, mt, nt);
      const int m0 = mt * BM, n0 = nt * BN;
      const int rows = min(BM, job.M - m0);
      if (!FWD && a_mn && p.cs.out && nt == 0 && slice == 0) sum_columns(p.cs, job.M, m0);
      const bool got = mbar_wait(&tfull[0], 0, abort_flag, p.err, kErrTimeoutEpilogue);
      const bool all_got = __all_sync(0xffffffffu, got);
      tc_fence_after_sync();
      float* part = reinterpret_cast<float*>(smem);
      if (all_got && quad * 32 < rows) {
        const uint32_t t_row = tmem_base + (static_cast<uint32_t>(quad * 32) << 16);
#pragma unroll 1
        for (int g = half; g < NG; g += 2) {
          uint32_t r[32];
          float v[32];
          tmem_ld32(t_row + g * 32, r);
          tmem_ld_wait(r);
#pragma unroll
          for (int j = 0; j < 32; ++j) v[j] = __uint_as_float(r[j]);
          if (quad * 32 + lane < rows) {
            float4* dst = reinterpret_cast<float4*>(part + (quad * 32 + lane) * T::PART_LD + g * 32);
#pragma unroll
            for (int q = 0; q < 8; ++q)
              dst[q] = make_float4(v[4 * q], v[4 * q + 1], v[4 * q + 2], v[4 * q + 3]);
          }
        }
      }
      __syncwarp();
      cluster_sync();
      if (ks == 2) finish_pieces<BN, FWD, 2>(e, part, slice, rows, m0, n0, job.N);
      else if (ks == 4) finish_pieces<BN, FWD, 4>(e, part, slice, rows, m0, n0, job.N);
      else finish_pieces<BN, FWD, 8>(e, part, slice, rows, m0, n0, job.N);
      __syncwarp();
      cluster_sync();  // no CTA leaves while another still reads its partial
    }
  }
  if (!PAIR && ks > 1 && warp == 0) {
    cluster_sync();
    cluster_sync();
  }
  tc_fence_before_sync();
  __syncthreads();
  if constexpr (PAIR) cluster_sync();  // neither CTA leaves while the other may signal its barriers
  if (warp == 1) {
    tc_fence_after_sync();
    if constexpr (PAIR) tmem_dealloc_pair(tmem_base, T::TMEM_COLS);
    else tmem_dealloc(tmem_base, T::TMEM_COLS);
  }
}

template <int BN, bool PAIR, LinearForm FORM>
cudaError_t launch_tile(const LinearPlan& plan, const LinearMaps& t, const Params& p, cudaStream_t s) {
  using T = Tile<BN, PAIR>;
  auto kern = k_linear<BN, PAIR, FORM>;
  static thread_local uint64_t ready = 0;  // devices on which the shared-memory limit is raised
  int dev = 0;
  if (cudaError_t e = cudaGetDevice(&dev)) return e;
  if (dev >= 64 || !(ready >> dev & 1u)) {
    if (cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, T::SMEM)) return e;
    if (dev < 64) ready |= uint64_t(1) << dev;
  }
  static_assert(T::RING == Tile<256, true>::RING, "the plan's number of stages takes one ring size");
  const unsigned span = PAIR ? 2u : static_cast<unsigned>(plan.ks);
  const int second = FORM == LINEAR_BOTH_GRADS ? 1 : 0;
  if (span == 1)
    return launch_pdl(kern, dim3(plan.grid), dim3(kThreads), T::SMEM, s, t.a[0], t.b[0], t.a[second], t.b[second], p, 1);
  return launch_pdl_cluster(kern, dim3(plan.grid), dim3(kThreads), T::SMEM, s, span, t.a[0], t.b[0], t.a[second], t.b[second], p,
                            PAIR ? 1 : plan.ks);
}

template <LinearForm FORM>
cudaError_t launch_form(const LinearPlan& plan, const LinearMaps& t, const Params& p, cudaStream_t s) {
  if constexpr (FORM == LINEAR_FORWARD_SWAPPED) {
    if (plan.bn == 16) return launch_tile<16, false, FORM>(plan, t, p, s);
    if (plan.bn == 32) return launch_tile<32, false, FORM>(plan, t, p, s);
  } else {
    if (plan.pair) {
      if constexpr (FORM == LINEAR_FORWARD) {
        if (plan.bn == 160) return launch_tile<160, true, FORM>(plan, t, p, s);
        if (plan.bn == 192) return launch_tile<192, true, FORM>(plan, t, p, s);
      }
      if (plan.bn == 128) return launch_tile<128, true, FORM>(plan, t, p, s);
      if (plan.bn == 256) return launch_tile<256, true, FORM>(plan, t, p, s);
      return cudaErrorInvalidValue;
    }
    if (plan.bn == 64) return launch_tile<64, false, FORM>(plan, t, p, s);
    if (plan.bn == 128) return launch_tile<128, false, FORM>(plan, t, p, s);
    if (plan.bn == 256) return launch_tile<256, false, FORM>(plan, t, p, s);
  }
  return cudaErrorInvalidValue;
}

// ---------------------------------------------------------------------------- a few rows
// y of a few rows: a warp takes an output feature at a time and streams its weights, 16
// bytes a lane, against the rows of x in shared memory.  The weights are read once and bound it:
// 42 MB for one row of 4608 x 4608.  Against the tensor-core kernel on a 128-row tile it needs no
// TMEM, clusters or partials, whose set-up is as long as the stream of a small layer.
constexpr int kFewThreads = 256;
constexpr int kFewSmem = 48 * 1024;

// F features a warp share what it reads of x.
template <int R, int F>
__global__ void __launch_bounds__(kFewThreads, F == 1 ? 4 : 2) k_linear_few(const __nv_bfloat16* x, int64_t ld_x, const __nv_bfloat16* w,
                                                            int64_t ld_w, int rows, int N, int K, const LinearEpilogue e) {
  // x in fp32, R rows of k8 pieces of 8; a piece's halves lie in two planes, so that the 16-byte
  // reads of a warp are contiguous
  extern __shared__ ulonglong2 sx[];
  const int lane = threadIdx.x & 31;
  const int k8 = K / 8, tail = K % 8;  // whole pieces, and elements behind them
  launch_dependents();
  const int first = (static_cast<int>(blockIdx.x) * (kFewThreads / 32) + (threadIdx.x >> 5)) * F;
  constexpr int UN = F == 1 ? 6 : 4;  // pieces of a feature in flight a lane
  grid_dependency_wait();
  // The first weights are on their way while x is staged.
  uint4 q[UN][F];
  auto fetch = [&](int f, int c) {
#pragma unroll
    for (int u = 0; u < UN; ++u)
#pragma unroll
      for (int j = 0; j < F; ++j)
        q[u][j] = reinterpret_cast<const uint4*>(w + static_cast<int64_t>(min(f + j, N - 1)) * ld_w)[c + u * 32];
  };
  bool fetched = first < N && lane + (UN - 1) * 32 < k8;
  if (fetched) fetch(first, lane);
  for (int i = threadIdx.x; i < R * k8; i += kFewThreads) {
    const int r = i / k8, c = i - r * k8;
    const uint4 q = r < rows ? reinterpret_cast<const uint4*>(x + r * ld_x)[c] : make_uint4(0, 0, 0, 0);
    sx[(2 * r) * k8 + c] = make_ulonglong2(bf16x2_f2(q.x), bf16x2_f2(q.y));
    sx[(2 * r + 1) * k8 + c] = make_ulonglong2(bf16x2_f2(q.z), bf16x2_f2(q.w));
  }
  __syncthreads();
  const int step = static_cast<int>(gridDim.x) * (kFewThreads / 32) * F;
  for (int f = first; f < N; f += step) {
    const uint4* wf[F];
#pragma unroll
    for (int j = 0; j < F; ++j) wf[j] = reinterpret_cast<const uint4*>(w + static_cast<int64_t>(min(f + j, N - 1)) * ld_w);
    uint64_t acc2[F][R] = {};
    auto piece = [&](const uint4 (&q)[F], int c) {
      uint64_t w2[F][4];
#pragma unroll
      for (int j = 0; j < F; ++j) {
        w2[j][0] = bf16x2_f2(q[j].x);
        w2[j][1] = bf16x2_f2(q[j].y);
        w2[j][2] = bf16x2_f2(q[j].z);
        w2[j][3] = bf16x2_f2(q[j].w);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const ulonglong2 lo = sx[(2 * r) * k8 + c], hi = sx[(2 * r + 1) * k8 + c];
#pragma unroll
        for (int j = 0; j < F; ++j) {
          acc2[j][r] = fma2(w2[j][0], lo.x, acc2[j][r]);
          acc2[j][r] = fma2(w2[j][1], lo.y, acc2[j][r]);
          acc2[j][r] = fma2(w2[j][2], hi.x, acc2[j][r]);
          acc2[j][r] = fma2(w2[j][3], hi.y, acc2[j][r]);
        }
      }
    };
    int c = lane;
    for (; c + (UN - 1) * 32 < k8; c += UN * 32) {
      if (!fetched) fetch(f, c);
      fetched = false;
#pragma unroll
      for (int u = 0; u < UN; ++u) piece(q[u], c + u * 32);
    }
    for (; c < k8; c += 32) {
      uint4 one[F];
#pragma unroll
      for (int j = 0; j < F; ++j) one[j] = wf[j][c];
      piece(one, c);
    }
    float acc[F][R];
#pragma unroll
    for (int j = 0; j < F; ++j)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float a, b;
        upk2(acc2[j][r], a, b);
        acc[j][r] = a + b;
      }
    if (lane < tail) {
#pragma unroll
      for (int j = 0; j < F; ++j) {
        const float wv = __bfloat162float(reinterpret_cast<const __nv_bfloat16*>(wf[j])[k8 * 8 + lane]);
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < rows) acc[j][r] = fmaf(wv, __bfloat162float(x[r * ld_x + k8 * 8 + lane]), acc[j][r]);
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
#pragma unroll
      for (int j = 0; j < F; ++j)
#pragma unroll
        for (int r = 0; r < R; ++r) acc[j][r] += __shfl_xor_sync(0xffffffffu, acc[j][r], o);
    // lane F r + j finishes feature j of row r
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int j = 0; j < F; ++j)
        if (lane == F * r + j) v = acc[j][r];
    const int row = lane / F, col = f + lane % F;
    if (row < rows && col < N) {
      if (e.bias) v += e.bias[col];
      if (e.z) e.z[row * e.ld_z + col] = __float2bfloat16_rn(v);
      float two[2] = {v, 0.0f};
      activate(two, e.act);
      v = two[0];
      if (e.residual) v += __bfloat162float(e.residual[row * e.ld_residual + col]);
      e.y[row * e.ld_y + col] = __float2bfloat16_rn(v);
    }
  }
}

template <int R, int F>
cudaError_t launch_few(const void* x, int64_t ld_x, const void* w, int64_t ld_w, int rows, int N, int K, const LinearEpilogue& e,
                       int sms, cudaStream_t s) {
  const int per = kFewThreads / 32 * F, grid = std::min((N + per - 1) / per, sms * 4);
  return launch_pdl(k_linear_few<R, F>, dim3(grid), dim3(kFewThreads), static_cast<size_t>(R) * (K / 8) * 32, s,
                    static_cast<const __nv_bfloat16*>(x), ld_x, static_cast<const __nv_bfloat16*>(w), ld_w, rows, N, K, e);
}

}  // namespace

// Up to four rows, as long as they fit shared memory and the sharing of x does not cost more than
// the tensor-core kernel's set-up (1 x 4608 x 4608: 9.5 us against 12.0 us; 2 rows 10.6 against 12.2;
// 4 rows of 1024 x 2816 4.1 against 5.0, of 2816 x 1024 5.9 against 5.3).  From two rows on, while the
// features take one round of the CTAs, 16 each, that the SMs hold at two: 2048 -> 4096 with 4 rows 6.8 against
// 7.6 us, 2048 -> 5632 10.2 against 8.1, 1824 -> 7656 17.0 against 8.9.  One row stays within 17 % of the other
// kernel wherever it is slower (1528 -> 12000: 11.4 against 9.9).
bool linear_is_few(int64_t M, int64_t N, int64_t K, int sms) {
  if (M == 1) return K * 4 <= kFewSmem;
  return N <= 32 * sms && (M == 2 ? M * K * 4 <= kFewSmem : (M <= 4 && K <= 2048));
}

cudaError_t launch_linear_few(const void* x, int64_t ld_x, const void* w, int64_t ld_w, int M, int N, int K, const LinearEpilogue& e,
                              int sms, cudaStream_t s) {
  if (M == 1) return launch_few<1, 1>(x, ld_x, w, ld_w, M, N, K, e, sms, s);
  if (M == 2) return launch_few<2, 2>(x, ld_x, w, ld_w, M, N, K, e, sms, s);
  return launch_few<4, 2>(x, ld_x, w, ld_w, M, N, K, e, sms, s);
}

namespace {

// Microseconds, fitted to every tile and split at 25 shapes of each form (1 to 8000 rows, widths 64
// to 4608): the plan with the least estimate runs within 0.9% of the fastest one on average there, 11% at
// worst; on 30 random shapes of each form that took no part in the fit, within 2.3% (forward), 1.8% (dx) and
// 0.8% (dW), 19% at worst, in launches of 3 to 25 us.  A stage takes the longest of its hand-over, its MMAs and its bytes into the SM; an
// epilogue runs under the next tile's stages where there is one; clusters stay inside a GPC, so
// that fewer of the larger ones fit (33 of 4 CTAs and 15 of 8, of 148 SMs).
// The pairs of 160 columns, which came after the fit, take the same constants; the swapped product has
// its own, from 48 shapes of 3 to 64 rows.
constexpr double kStart = 1.8, kPairStart = 0.87, kHandOver = 0.314, kMma = 0.035, kMmaColumn = 0.0011, kBytes = 132e3,
                 kEpilogue = 0.27, kColumn = 0.0207, kPlainColumn = 0.0074, kTile = 0.22, kPairTile = 0.75, kSplit = 1.48,
                 kSplitColumn = 0.0145, kSplitRank = 0.009, kSwapStage = 0.265, kSwapFinish = 0.25, kSwapSplit = 1.1, kSwapRow = 0.0385;
constexpr int kSwapRows = 32;  // at 64 columns the tile that holds them is as quick

// The tiles of a product D[M, N] over a contraction of K, and their times.
struct Tiling {
  int64_t tm, tn, tiles, kb;
  double stage, epilogue;
  Tiling(const LinearPlan& p, LinearForm form, int64_t M, int64_t N, int64_t K) {
    const int64_t bm = p.pair ? 2 * BM : BM;
    const int steps = linear_depth(p) / BK;
    tm = (M + bm - 1) / bm;
    tn = (N + p.bn - 1) / p.bn;
    tiles = tm * tn;
    kb = (K + linear_depth(p) - 1) / linear_depth(p);
    stage = std::max({kHandOver, steps * (kMma + kMmaColumn * p.bn), steps * (p.a_rows + (p.pair ? p.bn / 2 : p.bn)) * 128 / kBytes});
    // the two halves of the epilogue's warps take 32 columns in turn
    epilogue = kEpilogue + (form == LINEAR_FORWARD ? kColumn : kPlainColumn) * ((p.bn + 63) / 64 * 64);
  }
  // Time of all tiles on `slots` CTAs (pairs, clusters of ks).
  double time(const LinearPlan& p, int64_t slots, int ks, double finish) const {
    const int64_t waves = (tiles + slots - 1) / slots;
    const double main = stage * static_cast<double>((kb + ks - 1) / ks);
    return kStart + p.pair * kPairStart + main + (waves - 1) * (std::max(main, finish) + kTile + p.pair * kPairTile) + finish;
  }
};

// Pairs of 160 and 192 columns serve the forward, where fewer columns left over count for more than
// in the gradients, whose epilogue is short (784 x 1024 x 2816 with GELU: 12.5 us at 160 columns, 13.0
// at 192).
bool tile_exists(bool pair, int bn, LinearForm form) {
  const bool between = bn == 160 || bn == 192;
  return pair ? bn != 64 && (!between || form == LINEAR_FORWARD) : !between;
}

}  // namespace

LinearPlan plan_linear(LinearForm form, int64_t M, int64_t N, int64_t K, int sms) {
  LinearPlan best;
  for (int pair = 1; pair >= 0; --pair)
    for (int bn : {256, 192, 160, 128, 64}) {
      if (!tile_exists(pair, bn, form)) continue;
      LinearPlan p;
      p.pair = pair;
      p.bn = bn;
      p.a_rows = pair || form == LINEAR_WEIGHT_GRAD ? BM : static_cast<int>(std::min<int64_t>(BM, (M + 7) / 8 * 8));
      const Tiling t(p, form, M, N, K);
      if (t.tiles > (int64_t(1) << 30)) continue;
      for (int ks = 1; ks <= (pair ? 1 : 8); ks *= 2) {
        const int64_t slots = ks == 4 ? sms * 33 / 148 : (ks == 8 ? sms * 15 / 148 : sms / (pair ? 2 : ks));
        if (slots < 1 || (ks > 1 && (t.tiles > slots || t.kb < 2 * ks))) break;
        double finish = t.epilogue;
        if (ks > 1) finish = kSplit + (kSplitColumn + kSplitRank * ks) * bn * static_cast<double>(std::min<int64_t>(M, BM)) / BM;
        const double us = t.time(p, slots, ks, finish);
        if (best.bn && us >= best.us) continue;
        best = p;
        best.us = us;
        best.ks = ks;
        best.tiles_m[0] = static_cast<int>(t.tm);
        best.tiles_n[0] = static_cast<int>(t.tn);
        best.kb_total[0] = static_cast<int>(t.kb);
        best.grid = static_cast<int>(pair ? 2 * std::min(t.tiles, slots) : (ks > 1 ? t.tiles * ks : std::min(t.tiles, slots)));
      }
    }
  if (form != LINEAR_FORWARD || M > kSwapRows) return best;
  // A few rows as columns of D^T = W . x^T: the MMAs of a 128-feature tile then read 128 rows of weights
  // and 16 or 32 of x, where those of a 64-feature tile read 128 rows of x, existing or not (16 rows of
  // 256 -> 4608: 3.3 us against 4.3; of 2048 -> 12000: 11.7 against 14.0).
  LinearPlan p;
  p.swap = 1;
  p.bn = M <= 16 ? 16 : 32;
  p.a_rows = static_cast<int>(std::min<int64_t>(BM, (N + 7) / 8 * 8));
  const Tiling t(p, form, N, M, K);
  for (p.ks = 1; p.ks <= 2; ++p.ks) {
    if (t.tiles * p.ks > sms || (p.ks == 2 && t.kb < 4)) break;
    const double finish = p.ks == 1 ? kSwapFinish + kSwapRow * p.bn : kSwapSplit + kSwapRow * p.bn;
    p.us = kStart + kSwapStage * static_cast<double>((t.kb + p.ks - 1) / p.ks) + finish;
    if (p.us >= best.us) continue;
    best = p;
    best.tiles_m[0] = static_cast<int>(t.tm);
    best.tiles_n[0] = 1;
    best.kb_total[0] = static_cast<int>(t.kb);
    best.grid = static_cast<int>(t.tiles) * p.ks;
  }
  return best;
}

LinearPlan plan_linear_both(int64_t rows, int64_t in, int64_t out, int sms) {
  LinearPlan best;
  for (int pair = 1; pair >= 0; --pair)
    for (int bn : {256, 128, 64}) {
      if (!tile_exists(pair, bn, LINEAR_BOTH_GRADS)) continue;
      LinearPlan p;
      p.pair = pair;
      p.bn = bn;
      p.a_rows = BM;
      const Tiling x(p, LINEAR_BOTH_GRADS, rows, in, out), w(p, LINEAR_BOTH_GRADS, out, in, rows);
      if (x.tiles > (int64_t(1) << 30) || w.tiles > (int64_t(1) << 30)) continue;
      const int64_t slots = sms / (pair ? 2 : 1);
      // The input gradient in 1, 2, .. waves of its tiles, the weight gradient on the other CTAs.
      int64_t last = 0;
      for (int64_t waves = 1; waves <= 16; ++waves) {
        const int64_t ux = (x.tiles + waves - 1) / waves, uw = std::min(w.tiles, slots - ux);
        if (ux == last) break;
        last = ux;
        if (uw < 1) continue;
        const double us = std::max(x.time(p, ux, 1, x.epilogue), w.time(p, uw, 1, w.epilogue));
        if (best.bn && us >= best.us) continue;
        best = p;
        best.us = us;
        best.units = static_cast<int>(ux);
        best.grid = static_cast<int>((pair ? 2 : 1) * (ux + uw));
        const Tiling* t[2] = {&x, &w};
        for (int j = 0; j < 2; ++j) {
          best.tiles_m[j] = static_cast<int>(t[j]->tm);
          best.tiles_n[j] = static_cast<int>(t[j]->tn);
          best.kb_total[j] = static_cast<int>(t[j]->kb);
        }
      }
    }
  return best;
}

cudaError_t launch_linear(LinearForm form, const LinearPlan& plan, const LinearMaps& maps, const LinearProduct* products,
                          const ColumnSums& cs, uint32_t* err, cudaStream_t s) {
  Params p{};
  for (int j = 0; j < (form == LINEAR_BOTH_GRADS ? 2 : 1); ++j) {
    Job& job = p.job[j];
    job.M = products[j].M;
    job.N = products[j].N;
    job.e = products[j].e;
    job.tiles_m = plan.tiles_m[j];
    job.tiles_n = plan.tiles_n[j];
    job.kb_total = plan.kb_total[j];
  }
  p.units = plan.units;
  p.a_rows = plan.a_rows;
  p.stages = std::min(kMaxStages, Tile<256, true>::RING / (linear_depth(plan) * (plan.a_rows + (plan.pair ? plan.bn / 2 : plan.bn)) * 2));
  p.cs = cs;
  p.err = err;
  switch (form) {
    case LINEAR_FORWARD: return launch_form<LINEAR_FORWARD>(plan, maps, p, s);
    case LINEAR_FORWARD_SWAPPED: return launch_form<LINEAR_FORWARD_SWAPPED>(plan, maps, p, s);
    case LINEAR_INPUT_GRAD: return launch_form<LINEAR_INPUT_GRAD>(plan, maps, p, s);
    case LINEAR_WEIGHT_GRAD: return launch_form<LINEAR_WEIGHT_GRAD>(plan, maps, p, s);
    case LINEAR_BOTH_GRADS: return launch_form<LINEAR_BOTH_GRADS>(plan, maps, p, s);
  }
  return cudaErrorInvalidValue;
}

}  // namespace dsv4v
