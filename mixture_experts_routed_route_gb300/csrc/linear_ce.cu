// Softmax cross entropy of logits = scale h W^T over a large vocabulary
// without the logits in memory, and its gradient (moe_linear_ce_forward /
// _backward).
//
//   lse_t = log sum_v exp l_tv,   loss_t = lse_t - l_t,target + z lse_t^2
//   g_tv = dl_t ((1 + 2 z lse_t) softmax_tv - [v = target]) scale
//   dh = g W,   dW = g^T h
//
// Rows whose target is ignored take no part: the rows that count are packed
// into a copy of h (zeros up to a multiple of 256 rows), and every product
// runs over that many rows, read on the device.  So ignored tokens cost
// nothing, and what their rows of h hold (a NaN, infinities) reaches no sum.
//
// Products, on the tensor cores (tcgen05.mma kind::f16, BF16 operands, FP32
// accumulators), 256 x 256 output tiles on CTA pairs, one persistent launch
// each:
//   lse    h W^T:   a tile's epilogue keeps each row's maximum and sum of
//                   exponentials over its columns; a small kernel joins them
//   grad   h W^T again, for a piece of the vocabulary: the epilogue turns the
//                   logits into g, rounded to BF16
//   dh     g W:     W read MN-major; partial sums over the vocabulary in FP32,
//                   one store or one reduce-add by TMA a piece
//   dW     g^T h:   both operands read MN-major
// g is the one rounding between the accumulators and the results: 2^-8 at most,
// relative, as much as the results' own; where up to 64 rows count, what it
// leaves over takes part as well.  A factor that g's rows share (the 1 / N of a
// mean) is kept out of it, the `unit` m: g is formed as g / m and the results are
// multiplied by m in FP32.  With it inside, the target's g, near -dl scale in
// every row, is rounded the same way in all of them: of 255 to 2040 rows of equal
// weight all results were too large or too small by up to 0.0039.  m is the
// significand, 1 <= m < 2, of the largest finite |dl scale|, so that no exponent
// moves.
// Exponentials are in base 2 with one fused product, exp2(l k - m), k = scale
// log2 e: the rounding is relative to the small difference.
//
// What bounds it (one GB300).  Large products: the tensor cores under the power
// cap.  Forward 2048 x 7168 x 131072 2.13 to 2.3 ms (1.7 PFLOP/s), 4096 x 2048 x
// 131072 1.25 ms; backward 4096 x 2048 x 131072 3.9 to 4.2 ms, 1.57 to
// 1.69 PFLOP/s (three products, 6 T V D; floor 3.43 ms), 2048 x 7168 x 131072 7.0
// ms (1.65), 1531 x 1408 x 50021 with 30 % ignored 347 us (1.3; floor 235: the
// last of five row tiles holds 48 rows, the last of six column tiles 128).  One
// token: the weight's bytes, 90 us (6.0 TB/s; floor 79), backward 303 us (the
// weight read twice and its gradient written; floor 158: read once).  Small
// problems: the chain of launches, 6 to 9 us each beside their work (512 x 256 x
// 32768: forward 19 us, backward 50 us; floors 4.5 and 13.4).
// Larger pieces of the vocabulary are faster (launches, dh's sums): 4096 x 2048 x
// 131072 in pieces of 16384 entries 4.18 ms, 32768 3.94, 65536 3.79; pieces that
// stay in L2 are not.  Tried without gain: sixteen epilogue warps in the
// backward's products, rotated starts of the contraction.
//
// Warp roles: warp 0 TMA producer, warp 1 TMEM allocation and (rank 0) MMA
// issue for the pair, the other 8 or 16 epilogue (lane quadrant w % 4, a part of
// the tile's columns each).  A thread has its own row of the accumulator, so the
// softmax needs no exchange between threads.
#include <algorithm>

#include "kernels.cuh"
#include "moe_gb300.h"

namespace moe {

namespace {

constexpr int kTile = 256;         // rows and columns of a pair's tile
constexpr int kBk = 64;            // contraction elements a stage: 128 bytes
constexpr int kOperand = 128 * kBk * 2;
constexpr int kStage = 2 * kOperand;
enum CeKind { kLse, kGrad, kDh, kDw };

// E epilogue warps, 4 KB each to turn their values around (the forward: the
// warps' maxima and sums of a row).
template <int KIND, int E>
struct CeCfg {
  static constexpr int kThreads = 64 + 32 * E;
  static constexpr int kStages = 6;
  static constexpr int kTurn = KIND == kLse ? 16384 : E * 4096;
  static constexpr int kSmem = 1024 + kStages * kStage + kTurn + 256;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};
constexpr int kGroup = 8;          // row tiles that share the columns' operand before the next ones
// The tensor cores cut off, not round, at each of their additions, so a logit of
// 7168 elements is low by 7.5e-6 of itself in one sum (by 17e-6 where all products
// have one sign).  In the forward logits are therefore summed in segments, whose
// sums are added up in registers (segment_of; few tokens: 64 elements each, which
// costs them nothing), and of each row the one logit whose error does not show as
// a share of its result, the target's, is formed apart in both directions:
// pack_rows.  The backward's other logits are one sum: g is off by 1e-4 of itself
// at a logit of 10, its rounding 2^-9.
// Few tokens: at most 64, 32 a group of four epilogue warps.
constexpr int kFew = 64;
// Backward of at most so many rows that count: g in two parts, see product_rows.
constexpr int kTwice = 64;
constexpr int kFewSteps = 4;       // contraction steps of 64 a stage; each is a sum of its own
constexpr int kFewSmem = 228 * 1000;   // beside 3 KB that are static
static_assert(kFewSmem + 3 * 1024 <= 232448, "shared memory per CTA");
constexpr float kLog2e = 1.44269504f, kLn2 = 0.693147181f;
constexpr float kLowest = -1.0e30f;

// What the parts that the dh product sums apart are chosen from.
struct DhPlan {
  int D;
  int steps;             // stages of the contraction, a piece of the vocabulary
  int pairs;             // CTA pairs
  int rows;              // rows of partial sums that the workspace holds, of all parts
};

struct CeParams {
  const int* count;      // rows of the products, parts of dh, rows that count
  int rows_cap;          // their capacity, a multiple of 256
  int D, V;
  int v0, vn;            // piece of the vocabulary: first, number (backward)
  int first;             // dh: store (else add)
  int segment;           // lse: stages that one sum of a logit takes
  float k;               // scale log2 e
  const int* target;     // [rows_cap], -1 past the rows
  float2* part;          // lse: [column tiles, or CTAs][rows_cap]: maximum of l k, sum of exp2(l k - maximum)
  const float* hit;      // lse, grad: [rows_cap], l_target (before the scale) in FP32
  const float* lse2;     // grad: lse log2 e
  const float2* coef;    // grad: scale dl (1 + 2 z lse), scale dl
  const float* unit;     // backward: what g leaves out, and its reciprocal
  uint32_t* err;
};

__device__ __forceinline__ float exp2_fast(float x) {
  float r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
  return r;
}

// Both CTAs' loads of a stage complete on rank 0's barrier.
__device__ __forceinline__ void tma_load_2d_pair(void* smem_dst, const CUtensorMap* tm, uint32_t bar, int x, int y) {
  asm volatile(
      "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(y)
      : "memory");
}

// MN-major tile in the 128-byte swizzle: groups of 64 elements along M (or N),
// each 64 rows (contraction elements) of 128 bytes; 8-row atoms 1024 bytes
// apart along the contraction, groups 8 KB apart.
__device__ __forceinline__ uint64_t sdesc_mn_bf16(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(8192 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitTimeoutCycles / 8) return;
  }
}

// Parts of the vocabulary that the dh product sums apart, so that its tiles fill
// the pairs: what takes the least time by a stage's 0.27 us, a tile's 1.5 us
// around its stages, and the parts' sums at 4 TB/s (written once a piece, read in
// the end).  Chosen once a call for the rows that count, so on the device; every
// lane of a warp gets the number (1531 x 1408 x 50021 with 30 % ignored: the
// product planned for all tokens took 137 us, the call 358 instead of 343).
__device__ __forceinline__ int dh_parts(const DhPlan& d, int count) {
  const int rows = (count + kTile - 1) / kTile * kTile, tiles = rows / kTile * ((d.D + kTile - 1) / kTile);
  const float sums = static_cast<float>(count) * static_cast<float>(d.D) * 2.0e-6f;
  float least = 3.0e38f;
  int best = 1;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int s = 1 + (threadIdx.x & 31) + 32 * i;
    const float us = static_cast<float>((tiles * s + d.pairs - 1) / d.pairs) *
                         (0.27f * static_cast<float>((d.steps + s - 1) / s) + 1.5f) +
                     static_cast<float>(s) * sums;
    if (us < least && (s == 1 || (s <= d.steps && static_cast<long long>(s) * rows <= d.rows))) {
      least = us;
      best = s;
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    const float u = __shfl_xor_sync(0xFFFFFFFFu, least, o);
    const int b = __shfl_xor_sync(0xFFFFFFFFu, best, o);
    if (u < least || (u == least && b < best)) {
      least = u;
      best = b;
    }
  }
  return best;
}

// The products' sizes and the order of their tiles.
template <int KIND>
struct CeWork {
  int m, n;              // output rows and columns
  int mt, nt, total;
  int k, split_steps;    // contraction, stages of 64 of a split
  int splits;

  __device__ __forceinline__ CeWork(const CeParams& p, int rows) {
    m = KIND == kDw ? p.vn : rows;
    n = KIND == kLse ? p.V : KIND == kGrad ? p.vn : p.D;
    k = KIND == kDh ? p.vn : KIND == kDw ? rows : p.D;
    mt = (m + kTile - 1) / kTile;
    nt = (n + kTile - 1) / kTile;
    splits = KIND == kDh ? p.count[1] : 1;
    total = mt * nt * splits;
    split_steps = ((k + kBk - 1) / kBk + splits - 1) / splits;
  }
};
struct CeTile {
  int row0, col0, n, split, ks0, ks;
};
// Groups of kGroup row tiles; within one, column after column.
template <int KIND, int E>
__device__ __forceinline__ CeTile ce_tile(const CeWork<KIND>& w, int tile) {
  CeTile t;
  const int per = w.mt * w.nt;
  t.split = KIND == kDh ? tile / per : 0;
  int i = tile - t.split * per;
  const int g = i / (kGroup * w.nt);
  i -= g * kGroup * w.nt;
  const int rows = min(kGroup, w.mt - g * kGroup);
  const int c = i / rows;
  t.row0 = (g * kGroup + i - c * rows) * kTile;
  t.col0 = c * kTile;
  t.n = E == 8 && w.n - t.col0 <= 128 ? 128 : 256;
  t.ks0 = t.split * w.split_steps;
  t.ks = max(0, min(w.split_steps, (w.k + kBk - 1) / kBk - t.ks0));
  return t;
}

// 16 columns of the warp's 32 lanes: where 32 would not fit beside a row's sums.
__device__ __forceinline__ void tmem_ld16(uint32_t taddr, uint32_t (&r)[16]) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(taddr));
}

__device__ __forceinline__ void tmem_ld8(uint32_t taddr, uint32_t (&r)[8]) {
  asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
               : "r"(taddr));
}

// One 16-byte piece of a warp's 32 rows x 128 bytes, in the 128-byte swizzle.
__device__ __forceinline__ void stage16(uint8_t* ws, int lane, int piece, uint4 v) {
  *reinterpret_cast<uint4*>(ws + lane * 128 + ((piece ^ (lane & 7)) << 4)) = v;
}

__device__ __forceinline__ float max3(float a, float b, float c) {
  float r;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ unsigned long long pair_of(float a, float b) {
  unsigned long long r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ void split(unsigned long long v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ unsigned long long fma2(unsigned long long a, unsigned long long b, unsigned long long c) {
  unsigned long long r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Where a row's target is among its 32 logits, columns c .. c + 31: the logit in FP32.
__device__ __forceinline__ void take_target(float (&x)[32], int c, int row, int target, const CeParams& p) {
  if (static_cast<unsigned>(target - c) < 32u) {
    const float l = p.hit[row];
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (target - c == j) x[j] = l;
  }
}

// 32 logits of a row, columns c .. c + 31 of n, join its maximum and sum of exponentials.
__device__ __forceinline__ void join_chunk(float (&x)[32], int c, int n, int row, int target, const CeParams& p, float& top,
                                           float& sum) {
  if (c + 32 > n) {   // past the vocabulary
#pragma unroll
    for (int j = 0; j < 32; ++j)
      if (c + j >= n) x[j] = -INFINITY;
  }
  take_target(x, c, row, target, p);
  float m = x[0];
#pragma unroll
  for (int j = 1; j < 31; j += 2) m = max3(m, x[j], x[j + 1]);
  m = fmaxf(top, fmaxf(m, x[31]) * p.k);
  sum *= exp2_fast(top - m);
  top = m;
  unsigned long long s = pair_of(0.0f, 0.0f);
  const unsigned long long kk = pair_of(p.k, p.k), mm = pair_of(-m, -m);
#pragma unroll
  for (int j = 0; j < 32; j += 2) {
    float a, b;
    split(fma2(pair_of(x[j], x[j + 1]), kk, mm), a, b);
    s = add2(s, pair_of(exp2_fast(a), exp2_fast(b)));
  }
  float a, b;
  split(s, a, b);
  sum += a + b;
}

// SUMS: logits are summed in segments, p.segment stages each.
template <int KIND, int E, bool SUMS>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(CeCfg<KIND, E>::kThreads, 1)
    ce_gemm_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                   const __grid_constant__ CUtensorMap tmC, const CeParams p) {
  constexpr bool kAMn = KIND == kDw, kBMn = KIND == kDh || KIND == kDw;
  static_assert(!SUMS || (KIND == kLse && E == 16), "tiles of 256 columns, 64 a thread");
  constexpr int kStages = CeCfg<KIND, E>::kStages;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* turn = smem + kStages * kStage;    // [E warps][32 rows x 128 bytes]
  uint64_t* full = reinterpret_cast<uint64_t*>(turn + CeCfg<KIND, E>::kTurn);   // rank 0: both CTAs' operands landed
  uint64_t* empty = full + kStages;    // the stage's MMAs are done
  uint64_t* tfull = empty + kStages;   // [2] an accumulator is complete
  uint64_t* tempty = tfull + 2;        // [2] rank 0: both CTAs drained it
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  const int cid = blockIdx.x >> 1, ncl = gridDim.x >> 1;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * E);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch(&tmA);
    tma_prefetch(&tmB);
    if (KIND != kLse) tma_prefetch(&tmC);
  }
  if (warp == 1) {
    tmem_alloc_cg<2>(tmem_slot, 512);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  cluster_sync();   // the other CTA's barriers exist before anything arrives on them
  after_previous();
  const CeWork<KIND> w(p, *p.count);

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    uint32_t it = 0;
    bool ok = true;
    for (int tile = cid; ok && tile < w.total; tile += ncl) {
      const CeTile t = ce_tile<KIND, E>(w, tile);
      const int arow = t.row0 + 128 * rank;                                  // this CTA's rows of A
      const int brow = t.col0 + t.n / 2 * rank + (KIND == kGrad ? p.v0 : 0);   // its half of the N rows
      for (int ks = 0; ks < t.ks; ++ks, ++it) {
        const uint32_t slot = it % kStages, ph = (it / kStages) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&empty[slot], ph ^ 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* sa = smem + slot * kStage;
          uint8_t* sb = sa + kOperand;
          const uint32_t bar = cluster_addr(&full[slot], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * kStage);
          const int k0 = (t.ks0 + ks) * kBk;
          if constexpr (kAMn) {
            tma_load_2d_pair(sa, &tmA, bar, arow, k0);
            tma_load_2d_pair(sa + kOperand / 2, &tmA, bar, arow + 64, k0);
          } else {
            tma_load_2d_pair(sa, &tmA, bar, k0, arow);
          }
          if constexpr (kBMn) {
            const int kb = k0 + (KIND == kDh ? p.v0 : 0);
            tma_load_2d_pair(sb, &tmB, bar, brow, kb);
            tma_load_2d_pair(sb + kOperand / 2, &tmB, bar, brow + 64, kb);
          } else {
            tma_load_2d_pair(sb, &tmB, bar, k0, brow);
          }
        }
        __syncwarp();
      }
    }
    // no load of either CTA may still be landing when the cluster exits
    if (lane == 0 && rank == 0) {
      const uint32_t pend = it < static_cast<uint32_t>(kStages) ? it : static_cast<uint32_t>(kStages);
      for (uint32_t j = 0; j < pend; ++j) {
        const uint32_t i2 = it - 1 - j;
        drain_wait(&full[i2 % kStages], (i2 / kStages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ----------------------------------------------------- MMA issuer
      // BF16 operands, FP32 accumulators; bits 15, 16: A, B MN-major
      const uint32_t idesc0 = idesc_bf16(0, 256) | (kAMn ? kIdescAMnMajor : 0u) | (kBMn ? (1u << 16) : 0u);
      uint32_t it = 0, tc = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < w.total; tile += ncl) {
        const CeTile t = ce_tile<KIND, E>(w, tile);
        const uint32_t idesc = idesc0 | ((static_cast<uint32_t>(t.n) >> 3) << 17);
        // Sums of a tile, each in the accumulator whose turn it is; a loop of its own around the stages, which a test in
        // each of them slows down
        int ks = 0;
        for (bool more = true; more; more = SUMS && ks < t.ks) {
          const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
          ok = __all_sync(0xFFFFFFFFu, mbar_wait<true>(&tempty[acc], aph ^ 1, abort_flag, p.err));
          if (!ok) break;
          tc_fence_after();
          const uint32_t d_tmem = tmem + acc * 256;
          const int first = ks, end = SUMS ? min(t.ks, ks + p.segment) : t.ks;
          for (; ks < end; ++ks, ++it) {
            const uint32_t slot = it % kStages, ph = (it / kStages) & 1;
            ok = __all_sync(0xFFFFFFFFu, mbar_wait<true>(&full[slot], ph, abort_flag, p.err));
            if (!ok) break;
            tc_fence_after();
            if (lane == 0) {
              const uint32_t sa = smem_u32(smem + slot * kStage), sb = sa + kOperand;
#pragma unroll
              for (int j = 0; j < kBk / 16; ++j) {
                const uint64_t ad = kAMn ? sdesc_mn_bf16(sa + j * 2048) : sdesc_k_sw128(sa + j * 32);
                const uint64_t bd = kBMn ? sdesc_mn_bf16(sb + j * 2048) : sdesc_k_sw128(sb + j * 32);
                mma_bf16_pair(d_tmem, ad, bd, idesc, ((ks - first) | j) ? 1u : 0u);
              }
              tc_commit_pair_mc(&empty[slot], 3);
            }
            __syncwarp();
          }
          if (!ok) break;
          if (lane == 0) tc_commit_pair_mc(&tfull[acc], 3);
          __syncwarp();
          ++tc;
        }
      }
      if (lane == 0 && it > 0) {
        tc_commit_pair(drain);
        drain_wait(drain, 0);
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------- epilogue
    const int q = warp & 3, h = (warp - 2) >> 2;
    uint8_t* ws = turn + (warp - 2) * 4096;
    float2(*red)[E / 4][128] = reinterpret_cast<float2(*)[E / 4][128]>(turn);   // forward: [2 turns]
    const uint32_t tempty0 = cluster_addr(tempty, 0);
    uint32_t tc = 0;
    int side = 0;
    const int whole = KIND == kGrad ? p.count[2] : 0;
    const float unit = KIND == kGrad ? p.unit[1] : KIND == kDw ? p.unit[0] : 1.0f;
    bool dead = false;   // forward: a wait ran out of time; the tiles' barriers are still met
    struct {
      int target;
      float lse2;
      float2 coef;
    } next{};
    auto row_values = [&](int tile) {
      if constexpr (KIND == kLse || KIND == kGrad) {
        const int row = ce_tile<KIND, E>(w, tile).row0 + 128 * rank + 32 * q + lane;
        next.target = p.target[row];
        if constexpr (KIND == kGrad) {
          next.lse2 = p.lse2[row];
          next.coef = p.coef[row];
        }
      }
    };
    if (cid < w.total) row_values(cid);
    for (int tile = cid; tile < w.total; tile += ncl) {
      const CeTile t = ce_tile<KIND, E>(w, tile);
      const int row = t.row0 + 128 * rank + 32 * q + lane;     // this thread's
      const int row_w = row - lane;
      const int cols = t.n / (E / 4), c0 = t.col0 + h * cols;  // this warp's columns
      // Whether anything reads this warp's rows: those that count; of g, which the dW product reads 64 rows at a
      // time, those up to a multiple of 64; of dW, the vocabulary's.
      const bool live = KIND == kDw ? p.v0 + row_w < p.V : row_w < (KIND == kGrad ? (w.m + 63) / 64 * 64 : w.m);
      // what the rows need, asked for a tile ahead
      const int target = next.target - (KIND == kGrad ? p.v0 : 0);
      const float lse2 = next.lse2;
      const float2 coef = make_float2(next.coef.x * unit, next.coef.y * unit);
      const bool second = row >= whole;   // grad: what the rounding of the first row's g leaves over
      const bool seconds = KIND == kGrad && row_w + 31 >= whole && whole < w.m;
      if (tile + ncl < w.total) row_values(tile + ncl);
      // the accumulator whose turn it is: complete (false: a wait ran out of time), its first column, free again
      auto next_sum = [&] {
        const bool there =
            __all_sync(0xFFFFFFFFu, mbar_wait<true>(&tfull[tc & 1], (tc >> 1) & 1, abort_flag, p.err));
        tc_fence_after();
        return there;
      };
      auto sum_at = [&] { return tmem + (tc & 1) * 256 + h * cols + (static_cast<uint32_t>(q * 32) << 16); };
      auto sum_read = [&] {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * (tc & 1));
      };
      // this thread's columns: the sums of the segments, added up (false: a wait ran out of time)
      constexpr int kChunks = 32 / E;
      auto sum_up = [&](float (&x)[kChunks][32]) {
        for (int ks = 0; ks < t.ks; ks += p.segment, ++tc) {
          if (!next_sum()) return false;
          const uint32_t tbase = sum_at();
#pragma unroll
          for (int ci = 0; ci < kChunks; ++ci) {
#pragma unroll
            for (int i = 0; i < 32; i += 16) {
              uint32_t v[16];
              tmem_ld16(tbase + 32 * ci + i, v);
              tmem_ld_wait();
              if (i == 16 && ci == kChunks - 1) sum_read();
#pragma unroll
              for (int j = 0; j < 16; ++j)
                x[ci][i + j] = ks == 0 ? __uint_as_float(v[j]) : x[ci][i + j] + __uint_as_float(v[j]);
            }
          }
        }
        return true;
      };
      if constexpr (KIND == kLse) {
        float top = kLowest, sum = 0.0f;
        if constexpr (!SUMS) {
          dead = dead || !next_sum();
          const uint32_t tbase = sum_at();
#pragma unroll 1
          for (int ci = 0; ci < (dead ? 0 : cols / 32); ++ci) {
            uint32_t v[32];
            tmem_ld32(tbase + 32 * ci, v);
            tmem_ld_wait();
            if (ci == cols / 32 - 1) sum_read();   // every column has been read: the accumulator is free
            float x[32];
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
            join_chunk(x, c0 + 32 * ci, w.n, row, target, p, top, sum);
          }
          ++tc;
        } else {
          float x[kChunks][32];
          dead = dead || !sum_up(x);
#pragma unroll
          for (int ci = 0; ci < kChunks; ++ci)
            if (!dead) join_chunk(x[ci], c0 + 32 * ci, w.n, row, target, p, top, sum);
        }
        // the warps that share the rows
        red[side][h][32 * q + lane] = make_float2(top, sum);
        named_bar_sync(1 + q, 8 * E);
        if (h == 0) {
#pragma unroll
          for (int i = 1; i < E / 4; ++i) {
            const float2 r = red[side][i][32 * q + lane];
            const float m = fmaxf(top, r.x);
            sum = sum * exp2_fast(top - m) + r.y * exp2_fast(r.x - m);
            top = m;
          }
          p.part[static_cast<long long>(t.col0 / kTile) * p.rows_cap + row] = make_float2(top, sum);
        }
        side ^= 1;
      } else {
        if (!next_sum()) break;
        const uint32_t tbase = sum_at();
        if (!live) {
          sum_read();
          ++tc;
          continue;
        }
#pragma unroll 1
        for (int ci = 0; ci < cols / 32; ++ci) {
          uint32_t v[32];
          tmem_ld32(tbase + 32 * ci, v);
          tmem_ld_wait();
          if (ci == cols / 32 - 1) sum_read();   // every column has been read: the accumulator is free
          float x[32];
#pragma unroll
          for (int j = 0; j < 32; ++j) x[j] = __uint_as_float(v[j]);
          if (KIND != kGrad && t.ks == 0) {   // an empty contraction
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = 0.0f;
          }
          const int c = c0 + 32 * ci;
          constexpr int kHalves = KIND == kDh ? 1 : 2;   // chunks of 32 columns in 128 bytes
          if constexpr (KIND == kGrad) {
            take_target(x, c, row, target, p);
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] = coef.x * exp2_fast(fmaf(x[j], p.k, -lse2));
            if (static_cast<unsigned>(target - c) < 32u) {
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (target - c == j) x[j] -= coef.y;
            }
            if (c + 32 > w.n) {   // past the piece, whose end is the vocabulary's
#pragma unroll
              for (int j = 0; j < 32; ++j)
                if (c + j >= w.n) x[j] = 0.0f;
            }
            if (seconds) {
#pragma unroll
              for (int j = 0; j < 32; ++j) x[j] -= second ? __bfloat162float(__float2bfloat16_rn(x[j])) : 0.0f;
            }
          }
          if constexpr (KIND == kDw) {
#pragma unroll
            for (int j = 0; j < 32; ++j) x[j] *= unit;
          }
          if (ci % kHalves == 0) {   // the stores that read the buffer before are done
            if (lane == 0) bulk_wait_read<0>();
            __syncwarp();
          }
          if constexpr (KIND == kDh) {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              stage16(ws, lane, j, make_uint4(__float_as_uint(x[4 * j]), __float_as_uint(x[4 * j + 1]),
                                              __float_as_uint(x[4 * j + 2]), __float_as_uint(x[4 * j + 3])));
          } else {
#pragma unroll
            for (int j = 0; j < 4; ++j)
              stage16(ws, lane, 4 * (ci % kHalves) + j,
                      make_uint4(pack_bf16x2(x[8 * j], x[8 * j + 1]), pack_bf16x2(x[8 * j + 2], x[8 * j + 3]),
                                 pack_bf16x2(x[8 * j + 4], x[8 * j + 5]), pack_bf16x2(x[8 * j + 6], x[8 * j + 7])));
          }
          if (ci % kHalves == kHalves - 1) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
              const int cs = c - 32 * (kHalves - 1);
              if constexpr (KIND == kGrad) {
                tma_store_2d(&tmC, ws, cs, row_w);
              } else if constexpr (KIND == kDh) {
                if (cs < p.D) {
                  if (p.first) tma_store_2d(&tmC, ws, cs, t.split * w.mt * kTile + row_w);
                  else tma_reduce_add_2d(&tmC, ws, cs, t.split * w.mt * kTile + row_w);
                }
              } else {
                if (cs < p.D) tma_store_2d(&tmC, ws, cs, p.v0 + row_w);
              }
              bulk_commit();
            }
          }
        }
        ++tc;
      }
    }
    if (KIND != kLse && lane == 0) bulk_wait<0>();
    __syncwarp();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 1) tmem_dealloc_cg<2>(tmem, 512);
}

// Forward of at most N tokens: the vocabulary's rows are the products' rows, so
// that the tensor cores take N columns instead of 256 and what is left is the
// weight's one way from HBM.  A stage takes 512 bytes of a row at a time: with
// 128, the rows' neighbouring lines are asked for too far apart for HBM's pages
// (1 x 2048 x 131072 98.5 us, with 256 86.4, with 512 86.3).  Each CTA has a run
// of 32-row units, worked through in tiles of 128 rows (the last one shorter, and
// no row loaded twice); a thread keeps, for its place in the tiles, each token's
// running maximum and sum of exponentials, which lanes exchange once at the end.
template <int N>
__global__ void __launch_bounds__(64 + 4 * N, 1)
    ce_few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmH, const CeParams p) {
  constexpr int kStep = N * kBk * 2, kBytes = kFewSteps * (kOperand + kStep);
  constexpr int kFewStages = (kFewSmem - 1024 - 512) / kBytes;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kFewStages * kBytes);
  uint64_t* empty = full + kFewStages;
  uint64_t* tfull = empty + kFewStages;
  uint64_t* tempty = tfull + 2;
  uint64_t* drain = tempty + 2;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);
  __shared__ int targets[N];
  __shared__ float hits[N];
  __shared__ float2 red[4][N];

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  // this CTA's units of 32 rows
  const long long all = (p.V + 31) / 32;
  const int u0 = static_cast<int>(all * blockIdx.x / gridDim.x);
  const int units = static_cast<int>(all * (blockIdx.x + 1) / gridDim.x) - u0;
  const int tiles = (units + 3) / 4, steps = (p.D + kFewSteps * kBk - 1) / (kFewSteps * kBk);
  // the weight's rows of stage ks of a tile into slot `slot`
  auto load_w = [&](int tile, int ks, uint32_t slot) {
    const int n = min(4, units - 4 * tile);
    uint8_t* sa = smem + slot * kBytes;
    mbar_arrive_expect_tx(&full[slot], kFewSteps * (n * (32 * kBk * 2) + kStep));
    for (int i = 0; i < n; ++i)
#pragma unroll
      for (int j = 0; j < kFewSteps; ++j)
        tma_load_2d(sa + j * kOperand + i * (32 * kBk * 2), &tmW, &full[slot], (ks * kFewSteps + j) * kBk,
                    (u0 + 4 * tile + i) * 32);
  };
  const int ahead = min(tiles * steps, kFewStages);
  if (threadIdx.x == 0) {
    for (int s = 0; s < kFewStages; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], N / 8);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    // no kernel that may still run writes the weight: its first stages go out before the packed rows are waited for
    for (int i = 0; i < ahead; ++i) load_w(i / steps, i % steps, i);
    tma_prefetch(&tmH);
  }
  if (warp == 1) {
    tmem_alloc(tmem_slot, 2 * kFewSteps * N);
    tmem_relinquish();
  }
  after_previous();
  const int count = min(*p.count, N);
  if (threadIdx.x < N) {
    targets[threadIdx.x] = p.target[threadIdx.x];
    hits[threadIdx.x] = p.hit[threadIdx.x];   // anything past the rows that count, where the target is -1
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    uint32_t it = 0;
    bool ok = true;
    for (int tile = 0; ok && tile < tiles; ++tile) {
      for (int ks = 0; ks < steps; ++ks, ++it) {
        const uint32_t slot = it % kFewStages, ph = (it / kFewStages) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait(&empty[slot], ph ^ 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          if (it >= static_cast<uint32_t>(ahead)) load_w(tile, ks, slot);
#pragma unroll
          for (int j = 0; j < kFewSteps; ++j)
            tma_load_2d(smem + slot * kBytes + kFewSteps * kOperand + j * kStep, &tmH, &full[slot],
                        (ks * kFewSteps + j) * kBk, 0);
        }
        __syncwarp();
      }
    }
    // no load may still be landing when the CTA exits
    if (lane == 0) {
      const uint32_t pend = it < static_cast<uint32_t>(kFewStages) ? it : static_cast<uint32_t>(kFewStages);
      for (uint32_t j = 0; j < pend; ++j) {
        const uint32_t i2 = it - 1 - j;
        drain_wait(&full[i2 % kFewStages], (i2 / kFewStages) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    const uint32_t idesc = idesc_bf16(N, 128);
    uint32_t it = 0;
    bool ok = true;
    for (int tile = 0; ok && tile < tiles; ++tile) {
      for (int ks = 0; ks < steps; ++ks, ++it) {
        const uint32_t acc = it & 1, aph = (it >> 1) & 1, slot = it % kFewStages, ph = (it / kFewStages) & 1;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tempty[acc], aph ^ 1, abort_flag, p.err) &&
                                         mbar_wait(&full[slot], ph, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
        if (lane == 0) {
          const uint32_t sa = smem_u32(smem + slot * kBytes), sb = sa + kFewSteps * kOperand;
#pragma unroll
          for (int j = 0; j < kFewSteps * kBk / 16; ++j)   // a sum each 64 elements
            mma_bf16(tmem + (acc * kFewSteps + (j >> 2)) * N, sdesc_k_sw128(sa + (j >> 2) * kOperand + (j & 3) * 32),
                     sdesc_k_sw128(sb + (j >> 2) * kStep + (j & 3) * 32), idesc, (j & 3) ? 1u : 0u);
          tc_commit(&empty[slot]);
          tc_commit(&tfull[acc]);
        }
        __syncwarp();
      }
    }
    if (lane == 0 && it > 0) {
      tc_commit(drain);
      drain_wait(drain, 0);
    }
    __syncwarp();
  } else {
    const int q = warp & 3, j0 = 32 * ((warp - 2) >> 2);   // lane quadrant, tokens
    float top[32], sum[32];
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      top[j] = kLowest;
      sum[j] = 0.0f;
    }
    uint32_t it = 0;
    bool ok = true;
    for (int tile = 0; ok && tile < tiles; ++tile) {
      const int unit = 4 * tile + q, row = (u0 + unit) * 32 + lane;
      float x[32];
      for (int ks = 0; ks < steps; ++ks, ++it) {
        const uint32_t acc = it & 1, aph = (it >> 1) & 1;
        ok = __all_sync(0xFFFFFFFFu, mbar_wait(&tfull[acc], aph, abort_flag, p.err));
        if (!ok) break;
        tc_fence_after();
        const uint32_t at = tmem + acc * kFewSteps * N + j0 + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
        for (int i = 0; i < 32; i += 8) {   // the stage's sums in pairs
          uint32_t v[kFewSteps][8];
#pragma unroll
          for (int k = 0; k < kFewSteps; ++k) tmem_ld8(at + k * N + i, v[k]);
          tmem_ld_wait();
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const float s = (__uint_as_float(v[0][j]) + __uint_as_float(v[1][j])) +
                            (__uint_as_float(v[2][j]) + __uint_as_float(v[3][j]));
            x[i + j] = ks == 0 ? s : x[i + j] + s;
          }
        }
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&tempty[acc]);
      }
      if (!ok || unit >= units || row >= p.V) continue;
#pragma unroll
      for (int j = 0; j < 32; ++j) {
        if (j0 + j >= count) break;
        if (targets[j0 + j] == row) x[j] = hits[j0 + j];
        const float m = fmaxf(top[j], x[j] * p.k);
        sum[j] = fmaf(sum[j], exp2_fast(top[j] - m), exp2_fast(fmaf(x[j], p.k, -m)));
        top[j] = m;
      }
    }
    // over the warp's rows, and the warps'
#pragma unroll
    for (int j = 0; j < 32; ++j) {
      if (j0 + j >= count) break;
      float m = top[j];
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, o));
      float t = sum[j] * exp2_fast(top[j] - m);
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xFFFFFFFFu, t, o);
      if (lane == 0) red[q][j0 + j] = make_float2(m, t);
    }
    named_bar_sync(1, 4 * N);
    const int j = threadIdx.x - 64;
    if (j < count) {
      float m = red[0][j].x, t = red[0][j].y;
#pragma unroll
      for (int i = 1; i < 4; ++i) {
        const float2 r = red[i][j];
        const float n = fmaxf(m, r.x);
        t = t * exp2_fast(m - n) + r.y * exp2_fast(r.x - n);
        m = n;
      }
      p.part[static_cast<long long>(blockIdx.x) * p.rows_cap + j] = make_float2(m, t);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  if (warp == 1) tmem_dealloc(tmem, 2 * kFewSteps * N);
}

// ----------------------------------------------------- rows that count

struct RowParams {
  int T, D, V;
  int rows_cap;
  const void* targets;
  int wide;              // int64 targets
  long long ignore;
  const __nv_bfloat16* h;
  long long ldh;
  int* count;            // rows of the products, parts of dh, rows that count
  float* unit;           // backward: the factor that g leaves out, and its reciprocal
  DhPlan dh;             // backward
  int* list;             // [rows_cap] token of each packed row, -1 past them
  int* target;           // [rows_cap], -1 past them
  int* inv;              // [T] packed row of each token, -1 (backward)
  __nv_bfloat16* packed; // [rows_cap, D]
  // forward
  float* loss;
  float* lse;
  // backward
  const float* lse_in;
  const float* dloss;
  float scale, z;
  float* lse2;           // [rows_cap]
  float2* coef;          // [rows_cap]
  const __nv_bfloat16* weight;
  float* hit;            // [rows_cap] logit of each row's target
};

// Rows of the products.  The backward rounds g to BF16.  Of a few rows each
// result is one or a few products, so that a row's rounding shows in all of them
// (11 rows: results off by up to 0.0034 in norm, their own rounding 0.0017).  Few
// rows are therefore there twice: the first rows' g is rounded, the second rows' g
// is what that left over, to 2^-16 of g (the logits' own error aside).  The tiles
// are no more (1 x 2048 x 131072 300 and 305 us, 64 rows 297 and 307; 128 rows of
// 2048 x 32768 would take 119 instead of 99).  More rows are off by 0.0017 in norm
// where they share a weight, which the unit keeps out of g, and by 0.0023 where
// weights differ from row to row: a target's g of its own weight is then rounded
// by up to 2^-8, in rows of equal weight alike.
__device__ __forceinline__ int product_rows(const RowParams& p, int count) {
  return p.coef && count <= kTwice ? 2 * count : count;
}

// A turn of 1024 tokens from t0, of which `base` rows that count come before:
// the packed row of this thread's token (-1: it does not count) and its target,
// and the number of rows after the turn.  counts: the warps', a turn's own.  write: put
// down what the products need of the row, and keep in `most` the bits of this thread's largest finite |dl scale|;
// tokens that do not count get their results: loss 0 (NaN for a target outside the vocabulary), lse 0.
__device__ __forceinline__ int2 row_turn(const RowParams& p, int t0, int& base, int* counts, bool write, uint32_t& most) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int t = t0 + threadIdx.x;
  long long target = p.ignore;
  if (t < p.T) target = p.wide ? static_cast<const long long*>(p.targets)[t] : static_cast<const int*>(p.targets)[t];
  const bool on = target != p.ignore && target >= 0 && target < p.V;
  const unsigned vote = __ballot_sync(0xFFFFFFFFu, on);
  if (lane == 0) counts[warp] = __popc(vote);
  __syncthreads();
  const int mine = counts[lane];
  int before = 0, all = 0;
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    const int c = __shfl_sync(0xFFFFFFFFu, mine, i);
    if (i < warp) before += c;
    all += c;
  }
  const int at = base + before + __popc(vote & ((1u << lane) - 1));
  base += all;
  if (write) {
    if (on) {
      float lse = 0.0f, d = 0.0f;
      if (p.coef) {
        lse = p.lse_in[t];
        d = p.dloss[t] * p.scale;
        const uint32_t bits = __float_as_uint(d) & 0x7FFFFFFFu;
        if (bits < 0x7F800000u) most = max(most, bits);
      }
      // one turn: the second rows as well
      for (int i = at; i < (p.T <= 1024 ? product_rows(p, all) : at + 1); i += all) {
        p.list[i] = t;
        p.target[i] = static_cast<int>(target);
        if (p.coef) {
          p.lse2[i] = lse * kLog2e;
          p.coef[i] = make_float2(d * fmaf(2.0f * p.z, lse, 1.0f), d);
        }
      }
    } else if (t < p.T && p.loss) {
      p.loss[t] = target == p.ignore ? 0.0f : NAN;
      p.lse[t] = 0.0f;
    }
    if (t < p.T && p.inv) p.inv[t] = on ? at : -1;
  }
  return on ? make_int2(at, static_cast<int>(target)) : make_int2(-1, -1);
}

// After the last turn: the number of rows, the unit, the second rows, and what
// stands for none up to a multiple of 256.
__device__ __forceinline__ void row_end(const RowParams& p, int count, uint32_t most) {
  __shared__ uint32_t tops[32];
  const int rows = product_rows(p, count);
  if (p.coef) {
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if ((threadIdx.x & 31) == 0) tops[threadIdx.x >> 5] = most;
    __syncthreads();
    if (threadIdx.x < 32) {
      most = __reduce_max_sync(0xFFFFFFFFu, tops[threadIdx.x]);
      const float m = __uint_as_float((most & 0x007FFFFFu) | 0x3F800000u);
      if (threadIdx.x == 0) {
        p.unit[0] = m;
        p.unit[1] = 1.0f / m;
      }
    }
  }
  if (threadIdx.x < 32) {
    const int parts = p.inv ? dh_parts(p.dh, rows) : 1;
    if (threadIdx.x == 0) {
      p.count[0] = rows;
      p.count[1] = parts;
      p.count[2] = count;
    }
  }
  if (p.T > 1024 && rows > count) {
    __syncthreads();   // the rows are written down
    for (int i = count + threadIdx.x; i < rows; i += 1024) {
      p.list[i] = p.list[i - count];
      p.target[i] = p.target[i - count];
      p.lse2[i] = p.lse2[i - count];
      p.coef[i] = p.coef[i - count];
    }
  }
  const int end = (rows + kTile - 1) / kTile * kTile;
  for (int i = rows + threadIdx.x; i < end; i += 1024) {
    p.list[i] = -1;
    p.target[i] = -1;
    if (p.coef) {
      p.lse2[i] = 0.0f;
      p.coef[i] = make_float2(0.0f, 0.0f);
    }
  }
}

// Rows 0 .. end - 1 of the packed copy of h, row i that of the token row_at(i).x (-1: zeros), with its logit of the
// target row_at(i).y in FP32.  Where a token is confident, lse - l_target and softmax - 1 are differences of nearly equal numbers that show
// what the tensor cores cut off: at a logit of 40 and probability 0.9997 a sum of 7168 elements there was off by as much
// as the gradient.  It is the one entry of a row that cancels, so its logit alone is formed apart, the same way in both
// directions, while the row and the target's weights are at hand (1.3 us of a call on one token, 2 of one on 1072 rows).
// A row takes as many of the block's threads as it has pieces of eight elements (a power of two, warps at least), and the
// rows go round the blocks first.
template <typename RowAt>
__device__ __forceinline__ void pack_rows(const RowParams& p, int end, RowAt row_at) {
  __shared__ float sums[32];
  const int pieces = p.D / 8, block = blockDim.x;
  const int size = min(block, max(32, pieces > 1 ? 1 << (32 - __clz(pieces - 1)) : 1));
  const int groups = block / size, group = threadIdx.x / size, at = threadIdx.x - group * size;
  for (int i0 = blockIdx.x; i0 < end; i0 += gridDim.x * groups) {
    const int i = i0 + group * gridDim.x;
    const int2 row = i < end ? row_at(i) : make_int2(-1, -1);
    const int t = row.x;
    float s = 0.0f;
    if (i < end) {
      const __nv_bfloat16* in = p.h + static_cast<long long>(max(t, 0)) * p.ldh;
      uint4* out = reinterpret_cast<uint4*>(p.packed + static_cast<long long>(i) * p.D);
      const uint4* w = reinterpret_cast<const uint4*>(p.weight + static_cast<long long>(max(row.y, 0)) * p.D);
      for (int c = at; c < pieces; c += size) {
        uint4 v = make_uint4(0, 0, 0, 0);
        if (t >= 0) {
          if (p.ldh % 8 == 0) {
            v = reinterpret_cast<const uint4*>(in)[c];
          } else {
            const unsigned short* e = reinterpret_cast<const unsigned short*>(in) + 8 * c;
            v.x = e[0] | static_cast<uint32_t>(e[1]) << 16;
            v.y = e[2] | static_cast<uint32_t>(e[3]) << 16;
            v.z = e[4] | static_cast<uint32_t>(e[5]) << 16;
            v.w = e[6] | static_cast<uint32_t>(e[7]) << 16;
          }
          const uint4 u = w[c];
          float d = bf16_lo(v.x) * bf16_lo(u.x);
          d = fmaf(bf16_hi(v.x), bf16_hi(u.x), d);
          d = fmaf(bf16_lo(v.y), bf16_lo(u.y), d);
          d = fmaf(bf16_hi(v.y), bf16_hi(u.y), d);
          d = fmaf(bf16_lo(v.z), bf16_lo(u.z), d);
          d = fmaf(bf16_hi(v.z), bf16_hi(u.z), d);
          d = fmaf(bf16_lo(v.w), bf16_lo(u.w), d);
          s += fmaf(bf16_hi(v.w), bf16_hi(u.w), d);
        }
        out[c] = v;
      }
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
    if (size > 32) {   // the row's warps, in their order
      if ((threadIdx.x & 31) == 0) sums[threadIdx.x >> 5] = s;
      __syncthreads();
      if (at == 0) {
        s = 0.0f;
        for (int k = 0; k < size / 32; ++k) s += sums[(threadIdx.x >> 5) + k];
      }
      __syncthreads();   // before the next rows' sums
    }
    if (at == 0 && t >= 0) p.hit[i] = s;
  }
}

// Up to 1024 tokens: every block finds the rows that count, the first writes them down, and all pack them.
__global__ void __launch_bounds__(1024) ce_rows_once_kernel(const __grid_constant__ RowParams p) {
  __shared__ int counts[32];
  __shared__ int2 list[1024];
  // in this order: the forward of few tokens reads the weight before its own wait, and whatever ran before this call
  // has ended then
  wait_previous();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  int count = 0;
  uint32_t most = 0;
  const int2 mine = row_turn(p, 0, count, counts, blockIdx.x == 0, most);
  if (mine.x >= 0) list[mine.x] = make_int2(threadIdx.x, mine.y);
  if (blockIdx.x == 0) row_end(p, count, most);
  __syncthreads();
  const int rows = product_rows(p, count), end = (rows + kTile - 1) / kTile * kTile;
  pack_rows(p, end, [&](int i) { return i < rows ? list[i < count ? i : i - count] : make_int2(-1, -1); });
}

// More tokens: one block finds the rows, 1024 tokens a turn, and others pack them.
__global__ void __launch_bounds__(1024) ce_rows_kernel(const __grid_constant__ RowParams p) {
  __shared__ int counts[2][32];
  wait_previous();
  int base = 0;
  uint32_t most = 0;
  for (int t0 = 0, turn = 0; t0 < p.T; t0 += 1024, turn ^= 1) row_turn(p, t0, base, counts[turn], true, most);
  row_end(p, base, most);
}
__global__ void __launch_bounds__(256) ce_pack_kernel(const __grid_constant__ RowParams p) {
  after_previous();
  const int count = *p.count, end = (count + kTile - 1) / kTile * kTile;
  pack_rows(p, end, [&](int i) { return make_int2(p.list[i], p.target[i]); });
}

// loss and lse of the packed rows from the tiles' maxima and sums: 32 rows a
// block, 32 threads a row.
__global__ void __launch_bounds__(1024) ce_join_kernel(const float2* part, const float* hit, const int* list,
                                                       const int* count, int parts, int rows_cap, float k, float z,
                                                       float* loss, float* lse) {
  __shared__ float2 s[32][33];
  after_previous();
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int row = blockIdx.x * 32 + x, n = *count;
  if (static_cast<int>(blockIdx.x) * 32 >= n) return;
  float top = kLowest, sum = 0.0f;
  if (row < n) {
    for (int i0 = y; i0 < parts; i0 += 32 * 8) {
      float2 q[8];   // asked for together
#pragma unroll
      for (int j = 0; j < 8; ++j)
        q[j] = i0 + 32 * j < parts ? part[static_cast<long long>(i0 + 32 * j) * rows_cap + row] : make_float2(kLowest, 0.0f);
      float m = top;
#pragma unroll
      for (int j = 0; j < 8; ++j) m = fmaxf(m, q[j].x);
      sum *= exp2_fast(top - m);
#pragma unroll
      for (int j = 0; j < 8; ++j) sum = fmaf(q[j].y, exp2_fast(q[j].x - m), sum);
      top = m;
    }
  }
  s[y][x] = make_float2(top, sum);
  __syncthreads();
  // warp y joins row y's 32 sums
  const int r = blockIdx.x * 32 + y;
  if (r >= n) return;
  const float2 v = s[x][y];
  top = v.x;
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, o));
  sum = v.y * exp2_fast(v.x - top);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, o);
  if (x == 0) {
    // in base 2 until the end: the loss is rounded relative to itself
    const float ls = log2f(sum), l = (top + ls) * kLn2;
    const int t = list[r];
    lse[t] = l;
    loss[t] = fmaf(z * l, l, (fmaf(-hit[r], k, top) + ls) * kLn2);
  }
}

// dh: the sum of the splits' FP32 rows, times the unit, rounded; zeros for tokens
// that do not count.  A thread takes four columns and asks for four splits at a time.
__global__ void __launch_bounds__(256) ce_dh_kernel(const float* part, const int* count, const float* unit, const int* inv,
                                                    int T, int D, __nv_bfloat16* dh) {
  after_previous();
  const float m = *unit;
  const int n = count[0], splits = count[1], per = D / 4;
  const int parts = n > count[2] ? 2 * splits : splits;              // of the second rows as well
  const long long second = static_cast<long long>(count[2]) * D;
  const long long all = static_cast<long long>(T) * per, plane = static_cast<long long>((n + kTile - 1) / kTile * kTile) * D;
  const long long hop = static_cast<long long>(gridDim.x) * 256;
  for (long long k = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x; k < all; k += hop) {
    const int t = static_cast<int>(k / per), c = static_cast<int>(k - static_cast<long long>(t) * per) * 4;
    const int i = inv[t];
    float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    if (i >= 0) {
      const float* q = part + static_cast<long long>(i) * D + c;
      for (int s = 0; s < parts; s += 4) {
        float4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          v[j] = s + j < parts ? *reinterpret_cast<const float4*>(q + (s + j < splits ? (s + j) * plane
                                                                                      : (s + j - splits) * plane + second))
                               : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 4; ++j) a.x += v[j].x, a.y += v[j].y, a.z += v[j].z, a.w += v[j].w;
      }
    }
    *reinterpret_cast<uint2*>(dh + static_cast<long long>(t) * D + c) =
        make_uint2(pack_bf16x2(a.x * m, a.y * m), pack_bf16x2(a.z * m, a.w * m));
  }
}

// ------------------------------------------------------------------- host

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

bool config_ok(const moe_linear_ce_config* c) {
  if (!c || c->tokens < 0 || c->d_model < 1 || c->vocab < 1) return false;
  if (c->target_bytes != 4 && c->target_bytes != 8) return false;
  if (!(c->logit_scale > 0.0f) || c->logit_scale > 1.0e30f) return false;
  if (!(c->z_weight >= 0.0f) || c->z_weight > 1.0e30f) return false;
  return c->h_stride == 0 || c->h_stride >= c->d_model;
}
bool supported(const moe_linear_ce_config* c) {
  if (c->d_model % 8 != 0 || c->d_model > 65536 || c->vocab > (1 << 24) || c->tokens > (1 << 24)) return false;
  const long long row_tiles = (c->tokens + kTile - 1) / kTile, col_tiles = (c->vocab + kTile - 1) / kTile;
  return row_tiles * col_tiles < (1ll << 30);   // tiles are counted in 32 bits
}

// Tokens that the vocabulary-wise forward takes: the weight's bytes bound both,
// and it moves no others (1 x 2048 x 131072 87 and 103 us, 64 tokens 95 and 107).
bool few(int T) { return T <= kFew; }

struct Layout {
  int rows_cap, col_tiles;
  int64_t dh_rows;        // of partial sums
  int64_t piece;          // vocabulary entries a piece, a multiple of 256
  size_t count, unit, list, target, inv, lse2, coef, hit, part, packed, g, dh, bytes;
};
size_t take(size_t* at, size_t n) {
  const size_t r = *at;
  *at += (n + 255) / 256 * 256;
  return r;
}
Layout lay_out(const moe_linear_ce_config* c, bool backward, int64_t piece, int sms) {
  Layout l{};
  l.rows_cap = (c->tokens + kTile - 1) / kTile * kTile;
  l.col_tiles = (c->vocab + kTile - 1) / kTile;
  l.piece = std::min<int64_t>(piece, static_cast<int64_t>(l.col_tiles) * kTile);
  // 128 MB of partial sums, or one part of all rows
  l.dh_rows = std::max<int64_t>(l.rows_cap, std::min<int64_t>(64ll * l.rows_cap, (32 << 20) / c->d_model / kTile * kTile));
  const size_t rows = l.rows_cap, D = c->d_model;
  size_t at = 0;
  l.count = take(&at, 12);   // 256 bytes: the unit behind it
  l.unit = l.count + 16;
  l.list = take(&at, rows * 4);
  l.target = take(&at, rows * 4);
  l.packed = take(&at, rows * D * 2);
  l.hit = take(&at, rows * 4);
  if (backward) {
    l.inv = take(&at, rows * 4);
    l.lse2 = take(&at, rows * 4);
    l.coef = take(&at, rows * 8);
    l.dh = take(&at, static_cast<size_t>(l.dh_rows) * D * 4);
    l.g = take(&at, rows * 2 * l.piece);
  } else {
    // a column a tile, or for few tokens one a CTA; room for either, so that fewer tokens never want more
    l.part = take(&at, 8 * std::max(rows * l.col_tiles, c->tokens ? static_cast<size_t>(kTile) * sms : 0));
  }
  l.bytes = at;
  return l;
}

// 2D map of a row-major matrix, 128-byte boxes of `box_rows` rows.
bool map_2d(CUtensorMap* tm, const void* base, int64_t rows, int64_t cols, int box_rows, bool f32) {
  const int esz = f32 ? 4 : 2;
  const cuuint64_t dims[2] = {static_cast<cuuint64_t>(cols), static_cast<cuuint64_t>(rows)};
  const cuuint64_t strides[1] = {static_cast<cuuint64_t>(cols) * esz};
  const cuuint32_t box[2] = {static_cast<cuuint32_t>(128 / esz), static_cast<cuuint32_t>(box_rows)};
  return make_tmap_nd(tm, f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, base, dims, strides,
                      box, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int KIND, int E, bool SUMS = false>
cudaError_t launch_gemm_as(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const CeParams& p, int pairs,
                           long long tiles, cudaStream_t stream) {
  using C = CeCfg<KIND, E>;
  static PerDeviceOnce once;
  cudaError_t e = once.once([&] {
    return cudaFuncSetAttribute(ce_gemm_kernel<KIND, E, SUMS>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kSmem);
  });
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<CUtensorMap*>(&a), const_cast<CUtensorMap*>(&b), const_cast<CUtensorMap*>(&c),
                  const_cast<CeParams*>(&p)};
  const int grid = 2 * static_cast<int>(std::max<long long>(1, std::min<long long>(pairs, tiles)));
  return launch_dependent(reinterpret_cast<const void*>(ce_gemm_kernel<KIND, E, SUMS>), dim3(grid), C::kThreads, C::kSmem,
                          stream, args);
}
// Stages of 64 elements that one sum of a logit takes in the forward of more than
// kFew tokens: short enough that the loss is as good as torch's FP32 products make
// it (error in norm against 64 bits, and theirs: D 512 0.5e-6 and 0.5e-6, 1024 0.5
// and 0.75, 1408 0.85 and 0.9, 2048 1.0 and 1.2, 7168 1.0 and 2.5).  512 instead of
// 1024 elements a sum: 4096 x 1024 x 65536 416 and 390 us, 4096 x 2048 x 131072
// 1.30 and 1.23 ms.
int segment_of(int D) { return D <= 1024 ? 8 : 16; }

// Sixteen epilogue warps in the forward: eight do not hide the exponentials of a
// short product (512 x 256 x 32768 22.8 and 20.2 us, 4096 x 512 x 65536 224 and
// 210), and would have 128 columns of sums a thread to keep instead of 64, which
// spills (2048 x 7168 x 131072 2.39 and 2.25 ms).  The backward's products gained
// nothing.
template <int KIND>
cudaError_t launch_gemm(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& c, const CeParams& p, int pairs,
                        long long tiles, cudaStream_t stream) {
  if constexpr (KIND == kLse)
    return p.D > p.segment * kBk ? launch_gemm_as<KIND, 16, true>(a, b, c, p, pairs, tiles, stream)
                                 : launch_gemm_as<KIND, 16>(a, b, c, p, pairs, tiles, stream);
  else
    return launch_gemm_as<KIND, 8>(a, b, c, p, pairs, tiles, stream);
}

template <int N>
cudaError_t launch_few(const void* weight, const void* packed, const CeParams& p, int sms, cudaStream_t stream) {
  static PerDeviceOnce once;
  cudaError_t e = once.once(
      [&] { return cudaFuncSetAttribute(ce_few_kernel<N>, cudaFuncAttributeMaxDynamicSharedMemorySize, kFewSmem); });
  if (e != cudaSuccess) return e;
  CUtensorMap w, h;
  if (!map_2d(&w, weight, p.V, p.D, 32, false) || !map_2d(&h, packed, p.rows_cap, p.D, N, false))
    return cudaErrorInvalidValue;
  void* args[] = {&w, &h, const_cast<CeParams*>(&p)};
  return launch_dependent(reinterpret_cast<const void*>(ce_few_kernel<N>), dim3(sms), 64 + 4 * N, kFewSmem, stream, args);
}

cudaError_t launch_rows(const RowParams& p, int sms, cudaStream_t stream) {
  void* args[] = {const_cast<RowParams*>(&p)};
  if (p.T <= 1024)
    return launch_dependent(reinterpret_cast<const void*>(ce_rows_once_kernel), dim3(std::min(p.rows_cap, sms)), 1024, 0,
                            stream, args);
  const cudaError_t e = launch_dependent(reinterpret_cast<const void*>(ce_rows_kernel), dim3(1), 1024, 0, stream, args);
  if (e != cudaSuccess) return e;
  return launch_dependent(reinterpret_cast<const void*>(ce_pack_kernel), dim3(std::min(p.rows_cap, 8 * sms)), 256, 0,
                          stream, args);
}

template <typename X>
X* at(void* base, size_t off) {
  return reinterpret_cast<X*>(static_cast<uint8_t*>(base) + off);
}

// What the calls share: rows packed, parameters of the products.
void fill(const moe_linear_ce_config* c, const Layout& l, const void* h, const void* weight, const void* targets, void* ws,
          uint32_t* err, RowParams* r, CeParams* p) {
  r->T = c->tokens;
  r->D = c->d_model;
  r->V = c->vocab;
  r->rows_cap = l.rows_cap;
  r->targets = targets;
  r->wide = c->target_bytes == 8;
  r->ignore = c->ignore_index;
  r->h = static_cast<const __nv_bfloat16*>(h);
  r->ldh = c->h_stride ? c->h_stride : c->d_model;
  r->count = at<int>(ws, l.count);
  r->list = at<int>(ws, l.list);
  r->target = at<int>(ws, l.target);
  r->packed = at<__nv_bfloat16>(ws, l.packed);
  r->weight = static_cast<const __nv_bfloat16*>(weight);
  r->hit = at<float>(ws, l.hit);
  r->scale = c->logit_scale;
  r->z = c->z_weight;
  p->count = r->count;
  p->rows_cap = l.rows_cap;
  p->D = c->d_model;
  p->V = c->vocab;
  p->segment = segment_of(c->d_model);
  p->hit = r->hit;
  p->k = c->logit_scale * kLog2e;
  p->target = r->target;
  p->err = err;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_linear_ce_workspace_bytes(const moe_linear_ce_config* cfg, int backward, int32_t piece) {
  if (!config_ok(cfg) || !supported(cfg) || piece < 1) return 0;
  const int sms = device_sms();
  if (sms < 2) return 0;
  return lay_out(cfg, backward != 0, (static_cast<int64_t>(piece) + kTile - 1) / kTile * kTile, sms).bytes;
}

moe_status moe_linear_ce_forward(const moe_linear_ce_config* cfg, const void* h, const void* weight, const void* targets,
                                 float* loss, float* lse, void* workspace, size_t workspace_bytes,
                                 uint32_t* device_error_word, cudaStream_t stream) {
  if (!config_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!supported(cfg)) return MOE_ERR_UNSUPPORTED;
  if (cfg->tokens == 0) return MOE_OK;
  for (const void* q : {h, weight, targets, static_cast<const void*>(loss), static_cast<const void*>(lse)})
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return MOE_ERR_INVALID_ARG;
  if (!device_error_word || (reinterpret_cast<uintptr_t>(device_error_word) & 3)) return MOE_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (sms < 2) return MOE_ERR_CUDA;
  const Layout l = lay_out(cfg, false, kTile, sms);
  if (workspace_bytes < l.bytes) return MOE_ERR_CAPACITY;
  RowParams r{};
  CeParams p{};
  fill(cfg, l, h, weight, targets, workspace, device_error_word, &r, &p);
  r.loss = loss;
  r.lse = lse;
  p.part = at<float2>(workspace, l.part);
  if (launch_rows(r, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
  int parts = l.col_tiles;
  if (few(cfg->tokens)) {
    parts = sms;
    if ((cfg->tokens <= 32 ? launch_few<32>(weight, r.packed, p, sms, stream)
                           : launch_few<64>(weight, r.packed, p, sms, stream)) != cudaSuccess)
      return MOE_ERR_CUDA;
  } else {
    CUtensorMap a, b;
    if (!map_2d(&a, r.packed, l.rows_cap, cfg->d_model, 128, false) ||
        !map_2d(&b, weight, cfg->vocab, cfg->d_model, 128, false) ||
        launch_gemm<kLse>(a, b, a, p, sms / 2, static_cast<long long>(l.rows_cap / kTile) * l.col_tiles, stream) !=
            cudaSuccess)
      return MOE_ERR_CUDA;
  }
  float k = p.k, z = cfg->z_weight;
  const float2* part = p.part;
  const float* hit = p.hit;
  const int* list = r.list;
  const int* count = r.count;
  int cap = l.rows_cap;
  void* args[] = {&part, &hit, &list, &count, &parts, &cap, &k, &z, &loss, &lse};
  if (launch_dependent(reinterpret_cast<const void*>(ce_join_kernel), dim3((cfg->tokens + 31) / 32), 1024, 0, stream,
                       args) != cudaSuccess)
    return MOE_ERR_CUDA;
  return MOE_OK;
}

moe_status moe_linear_ce_backward(const moe_linear_ce_config* cfg, const void* h, const void* weight, const void* targets,
                                  const float* lse, const float* d_loss, void* dh, void* dweight, void* workspace,
                                  size_t workspace_bytes, uint32_t* device_error_word, cudaStream_t stream) {
  if (!config_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!supported(cfg)) return MOE_ERR_UNSUPPORTED;
  const int T = cfg->tokens, D = cfg->d_model, V = cfg->vocab;
  if (T == 0) {   // no rows: the weight's gradient is zero
    if (!aligned16(dweight)) return MOE_ERR_INVALID_ARG;
    return !dweight || cudaMemsetAsync(dweight, 0, 2ull * V * D, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  for (const void* q : {h, weight, targets, static_cast<const void*>(lse), static_cast<const void*>(d_loss)})
    if (!q || !aligned16(q)) return MOE_ERR_INVALID_ARG;
  if ((!dh && !dweight) || !aligned16(dh) || !aligned16(dweight)) return MOE_ERR_INVALID_ARG;
  if (!workspace || (reinterpret_cast<uintptr_t>(workspace) & 255)) return MOE_ERR_INVALID_ARG;
  if (!device_error_word || (reinterpret_cast<uintptr_t>(device_error_word) & 3)) return MOE_ERR_INVALID_ARG;
  const int sms = device_sms();
  if (sms < 2) return MOE_ERR_CUDA;
  // the largest pieces that the workspace holds
  Layout l = lay_out(cfg, true, kTile, sms);
  if (workspace_bytes < l.bytes) return MOE_ERR_CAPACITY;
  const size_t more = (workspace_bytes - l.bytes) / (static_cast<size_t>(l.rows_cap) * 2 * kTile);
  const int64_t most = static_cast<int64_t>(std::min<size_t>(more + 1, l.col_tiles));   // tiles of 256 entries a piece
  const int64_t pieces = (l.col_tiles + most - 1) / most;
  l = lay_out(cfg, true, (l.col_tiles + pieces - 1) / pieces * kTile, sms);
  RowParams r{};
  CeParams p{};
  fill(cfg, l, h, weight, targets, workspace, device_error_word, &r, &p);
  r.lse_in = lse;
  r.dloss = d_loss;
  r.inv = at<int>(workspace, l.inv);
  r.lse2 = at<float>(workspace, l.lse2);
  r.coef = at<float2>(workspace, l.coef);
  p.lse2 = r.lse2;
  p.coef = r.coef;
  r.unit = at<float>(workspace, l.unit);
  p.unit = r.unit;
  r.dh = {D, static_cast<int>(l.piece / kBk), sms / 2, static_cast<int>(l.dh_rows)};
  __nv_bfloat16* g = at<__nv_bfloat16>(workspace, l.g);
  float* part = at<float>(workspace, l.dh);
  CUtensorMap hk, hm, wk, wm, gk, gm, gs, ds, os;
  if (!map_2d(&hk, r.packed, l.rows_cap, D, 128, false) || !map_2d(&hm, r.packed, l.rows_cap, D, 64, false) ||
      !map_2d(&wk, weight, V, D, 128, false) || !map_2d(&wm, weight, V, D, 64, false) ||
      !map_2d(&gk, g, l.rows_cap, l.piece, 128, false) || !map_2d(&gm, g, l.rows_cap, l.piece, 64, false) ||
      !map_2d(&gs, g, l.rows_cap, l.piece, 32, false) ||
      !map_2d(&os, part, l.dh_rows, D, 32, true) ||
      (dweight && !map_2d(&ds, dweight, V, D, 32, false)))
    return MOE_ERR_CUDA;
  if (launch_rows(r, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
  const long long row_tiles = l.rows_cap / kTile, d_tiles = (D + kTile - 1) / kTile;
  for (int64_t v0 = 0; v0 < V; v0 += l.piece) {
    p.v0 = static_cast<int>(v0);
    p.vn = static_cast<int>(std::min<int64_t>(l.piece, V - v0));
    p.first = v0 == 0;
    const long long v_tiles = (p.vn + kTile - 1) / kTile;
    if (launch_gemm<kGrad>(hk, wk, gs, p, sms / 2, row_tiles * v_tiles, stream) != cudaSuccess) return MOE_ERR_CUDA;
    if (dh && launch_gemm<kDh>(gk, wm, os, p, sms / 2, sms / 2, stream) != cudaSuccess)
      return MOE_ERR_CUDA;
    if (dweight && launch_gemm<kDw>(gm, hm, ds, p, sms / 2, v_tiles * d_tiles, stream) != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (dh) {
    int t = T, d = D;
    const float* in = part;
    const int* inv = r.inv;
    __nv_bfloat16* out = static_cast<__nv_bfloat16*>(dh);
    const int* count = r.count;
    const float* unit = r.unit;
    void* args[] = {&in, &count, &unit, &inv, &t, &d, &out};
    const long long blocks = (static_cast<long long>(T) * (D / 4) + 255) / 256;
    if (launch_dependent(reinterpret_cast<const void*>(ce_dh_kernel),
                         dim3(static_cast<unsigned>(std::min<long long>(blocks, 16 * sms))), 256, 0, stream,
                         args) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
