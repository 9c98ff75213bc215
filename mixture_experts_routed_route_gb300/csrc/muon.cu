// Weight updates made orthogonal by Newton-Schulz products
// (moe_orthogonalize, moe_muon_update), for stacked matrices [E, rows, cols].
//
// One step on X (the smaller of rows and cols is m, the larger k):
//   wide (rows <= cols):  A = X X^T,  B = b A + c A A,  X <- a X + B X
//   tall (rows >  cols):  A = X^T X,  B = b A + c A A,  X <- a X + X B
// from X = U / (|U|_F + eps).  In exact arithmetic both are the polynomial
// a s + b s^3 + c s^5 of every singular value s of X.
//
// Numbers.  The products run on the tensor cores (tcgen05.mma kind::f16,
// FP16 operands, FP32 accumulators).  X itself is kept to 22 bits as two
// FP16 halves, hi + lo, of which the products read hi alone, and the
// diagonal of B is kept in FP32 and applied to hi + lo in the epilogue
// (B's FP16 copy has zeros there).  Why: a gradient is a few strong
// directions over a weak full-rank part, and five steps magnify the weak
// part up to 485 times.  Rounding X between the steps to FP16 spreads
// 2^-12 of the strong part over all directions, where it is magnified as
// well (1.6e-2 of the result's norm on rank 16 + 2 % noise; BF16: 1.3e-1);
// with X kept, the rounding of hi inside the products is projected onto the
// strong directions by B and does not grow (2e-4).  The diagonal matters in
// the other regime, X near orthogonal: there A is close to a multiple of
// the identity, and one rounding of B's almost equal diagonal entries
// scales the whole of X (Gaussian matrices: 1.6e-3 without, 7e-4 with).
// X is stored times 2^12, A and B times 2^9 (exact powers of two), so that
// FP16 keeps its 11 bits down to elements of 1.5e-8 of X and 1.2e-7 of A and
// B (with 2^11 for these the errors above are the same to three digits), and
// has room for elements of X up to 15.9, of A up to 127 (X's singular values
// up to 11, as A_ij <= s^2) and of B off its diagonal up to 127 (half the
// spread of B's eigenvalues b s^2 + c s^4 at most).
//
// Matrices with m <= 256 may go through all steps in one launch instead
// (muon_small.cu).  Otherwise each product is one persistent launch over
// 256 x 256 output tiles of all matrices, a tile on a CTA pair (cta_group::2, M = 256, N = 256: per SM a
// stage of 128 contraction elements is 64 KB of operands for 2 x 256 x 256 x
// 128 flops on the pair).  A and B are symmetric: only tiles on or above
// the diagonal are computed, and their epilogue stores the mirror image too.
// Tall and wide matrices need no transposes: the operand whose contraction
// index is not the fastest one in memory is read MN-major by the same tensor
// map (64-column chunks as an axis of their own).
//
// What bounds it.  Large matrices: operands and epilogues together draw about
// 14 TB/s from L2.  8 x 7168 x 2048, 3.05 ms, is 1.3 PFLOP/s over the call and
// 1.5 over its products (the Gram product 1.6, the apply products 1.5 with 315
// us each), where a library product reaches 1.7 in a long run under the power
// cap.  64 x 1408 x 2048 with the momentum and a float32 weight, 5.25 ms: the
// products run at 1.06 PFLOP/s (4.5 ms, 11.6 us an apply tile of 11 stages; no
// counters were taken at this shape), momentum and start kernels take 0.54 ms
// and the weight 0.25 ms of the last product; a BF16 weight 5.2 ms.
// Stacks in several runs of matrices: 96 x 7168 x 2048 39 ms, its step 42 ms.
// Small ones (3 x 1000 x 1531, 209 us): the chain of 15 dependent launches of
// 10 to 28 us each.
//
// Warp roles: warp 0 TMA producer, warp 1 TMEM allocation and (rank 0) MMA
// issue for the pair, warps 2 .. 9 epilogue (lane quadrant w % 4; every other
// 32 columns of the tile, or, of X, every other 64 in two halves of the rows).
// What a chunk reads besides the accumulator is asked for one chunk ahead, over
// the tile's end too: the update of 64 x 1408 x 2048 790 to 722 us.  Both
// CTAs' loads complete on rank 0's barrier of the stage.
#include <algorithm>
#include <atomic>
#include <cmath>

#include "moe_gb300_testing.h"
#include "muon_core.cuh"

namespace moe {

namespace {

// The error word of callers without one of their own: a device's copy is zero
// from the library's load on, so a first call may be inside a graph capture.
__device__ uint32_t g_error_word;

// Tile of BN = 256 or 128 columns (256 rows on the pair): stages of 128
// contraction elements, in two 64-element chunks of 128 (A) and BN / 2 (B)
// rows per CTA; 4 KB an epilogue warp to turn its 32 x 32 chunks around.
template <int BN>
struct NsCfg {
  static constexpr int kA = 2 * 128 * 128, kB = 2 * (BN / 2) * 128;
  static constexpr int kStage = kA + kB;
  static constexpr int kStages = BN == 256 ? 3 : 4;
  static constexpr int kSmem = 1024 + kStages * kStage + kEpiWarps * 4096 + 256;
  static_assert(kSmem <= 232448, "shared memory per CTA");
};

// Symmetric outputs: row q of 256 rows has the column tiles from its first
// one on.
template <int KIND, int BN>
__device__ __forceinline__ NsTile ns_tile(const NsParams& p, int tile, int rank) {
  NsTile t;
  t.mat = tile / p.tiles;
  int i = tile - t.mat * p.tiles, q = 0;
  if (KIND == kGram || KIND == kPoly) {
    constexpr int kPer = 256 / BN;
    for (; i >= p.col_tiles - q * kPer; ++q) i -= p.col_tiles - q * kPer;
    i += q * kPer;
  } else {
    q = i / p.col_tiles;
    i -= q * p.col_tiles;
  }
  t.row0 = q * 256 + 128 * rank;
  t.col0 = i * BN;
  t.n = (BN == 256 && p.valid_cols - t.col0 <= 128) ? 128 : BN;
  return t;
}

// Chunk ci of epilogue warp (q, h).
template <int KIND>
__device__ __forceinline__ NsChunk ns_chunk_of(const NsTile& t, int q, int h, int ci) {
  NsChunk k;
  k.half = KIND >= kApply ? ci & 1 : 0;
  k.tcol = KIND >= kApply ? 64 * (h + 2 * (ci >> 1)) : 32 * (h + 2 * ci);
  k.row = t.row0 + 32 * q + 16 * k.half;
  k.col = t.col0 + k.tcol;
  return k;
}

template <int KIND, int BN>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
              const __grid_constant__ CUtensorMap tmLo, const NsParams p) {
  using C = NsCfg<BN>;
  constexpr int kStages = C::kStages, kStageBytes = C::kStage;
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  float* turn = reinterpret_cast<float*>(smem + kStages * kStageBytes);   // [8 warps][32 x 32]
  uint64_t* full = reinterpret_cast<uint64_t*>(turn + kEpiWarps * 1024);   // rank 0: both CTAs' operands landed
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
      mbar_init(&tempty[a], 2 * kEpiWarps);
    }
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch(&tmA);
    tma_prefetch(&tmB);
  }
  if (warp == 1) {
    tmem_alloc_cg<2>(tmem_slot, 2 * BN);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  cluster_sync();   // the other CTA's barriers exist before anything arrives on them
  after_previous();
  int total = p.total;
  if constexpr (KIND >= kFinal) {
    // unfinished products: the caller's tensors stay as they are
    const uint32_t lost = *p.lost;
    if (lost != 0) {
      total = 0;
      if (blockIdx.x == 0 && threadIdx.x == 0) atomicOr(p.err, lost);
    }
  }

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    uint32_t it = 0;
    bool ok = true;
    for (int tile = cid; ok && tile < total; tile += ncl) {
      const NsTile t = ns_tile<KIND, BN>(p, tile, rank);
      const int brow = t.col0 + t.n / 2 * rank;   // this CTA's half of the N rows
      const int ks_all = p.split ? 2 * p.kstages : p.kstages;
      for (int ks = 0; ks < ks_all; ++ks, ++it) {
        const uint32_t slot = it % kStages, ph = (it / kStages) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&empty[slot], ph ^ 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* sa = smem + slot * kStageBytes;
          const uint32_t bar = cluster_addr(&full[slot], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * kStageBytes);
          const bool low = ks >= p.kstages;   // X, the A operand if tall, is its lo half
          const int k0 = (low ? ks - p.kstages : ks) * 128;
          const CUtensorMap* ta = low && p.diag_cols ? &tmLo : &tmA;
          const CUtensorMap* tb = low && !p.diag_cols ? &tmLo : &tmB;
          if (p.a_mn) tma_load_4d_pair(sa, ta, bar, 0, k0, t.row0 >> 6, t.mat);
          else tma_load_4d_pair(sa, ta, bar, 0, t.row0, k0 >> 6, t.mat);
          if (p.b_mn) tma_load_4d_pair(sa + C::kA, tb, bar, 0, k0, brow >> 6, t.mat);
          else tma_load_4d_pair(sa + C::kA, tb, bar, 0, brow, k0 >> 6, t.mat);
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
      // FP16 operands (formats 0), FP32 accumulators; bits 15, 16: A, B MN-major
      const uint32_t idesc0 = (1u << 4) | ((256u >> 4) << 24) | (p.a_mn ? kIdescAMnMajor : 0u) | (p.b_mn ? (1u << 16) : 0u);
      uint32_t it = 0, tc = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < total; tile += ncl, ++tc) {
        const uint32_t idesc = idesc0 | ((static_cast<uint32_t>(ns_tile<KIND, BN>(p, tile, rank).n) >> 3) << 17);
        const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&tempty[acc], aph ^ 1, abort_flag, p.err))) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * BN;
        const int ks_all = p.split ? 2 * p.kstages : p.kstages;
        for (int ks = 0; ks < ks_all; ++ks, ++it) {
          const uint32_t slot = it % kStages, ph = (it / kStages) & 1;
          if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&full[slot], ph, abort_flag, p.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t sa = smem_u32(smem + slot * kStageBytes), sb = sa + C::kA;
#pragma unroll
            for (int j = 0; j < 8; ++j) {   // 16 contraction elements each
              const uint64_t ad = p.a_mn ? sdesc_mn_f16(sa + j * 2048) : sdesc_k_sw128(sa + (j >> 2) * 16384 + (j & 3) * 32);
              const uint64_t bd = p.b_mn ? sdesc_mn_f16(sb + j * 2048) : sdesc_k_sw128(sb + (j >> 2) * (C::kB / 2) + (j & 3) * 32);
              mma_bf16_pair(d_tmem, ad, bd, idesc, (ks | j) ? 1u : 0u);
            }
            tc_commit_pair_mc(&empty[slot], 3);
          }
          __syncwarp();
        }
        if (!ok) break;
        if (lane == 0) tc_commit_pair_mc(&tfull[acc], 3);
        __syncwarp();
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
    constexpr int kChunks = BN / 64;     // of 32 columns, per warp
    float* ws = turn + (warp - 2) * 1024;
    const uint32_t tempty0 = cluster_addr(tempty, 0);
    uint32_t tc = 0;
    ChunkIn<KIND> in;   // of the chunk at hand, from one chunk before it (of the tile before) on
    if (cid < total) {
      const NsTile t = ns_tile<KIND, BN>(p, cid, rank);
      const NsChunk k = ns_chunk_of<KIND>(t, q, h, 0);
      load_chunk_in(p, t.mat, k.row, k.col, lane, in);
    }
    for (int tile = cid; tile < total; tile += ncl, ++tc) {
      const NsTile t = ns_tile<KIND, BN>(p, tile, rank);
      const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
      auto load_next = [&](int ci) {
        if (ci + 1 < kChunks) {
          const NsChunk k = ns_chunk_of<KIND>(t, q, h, ci + 1);
          load_chunk_in(p, t.mat, k.row, k.col, lane, in);
        } else if (tile + ncl < total) {
          const NsTile tn = ns_tile<KIND, BN>(p, tile + ncl, rank);
          const NsChunk k = ns_chunk_of<KIND>(tn, q, h, 0);
          load_chunk_in(p, tn.mat, k.row, k.col, lane, in);
        }
      };
      if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&tfull[acc], aph, abort_flag, p.err))) break;
      tc_fence_after();
      const uint32_t tbase = tmem + acc * BN + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
      for (int ci = 0; ci < kChunks; ++ci) {
        const NsChunk k = ns_chunk_of<KIND>(t, q, h, ci);
        // a symmetric output's blocks below the diagonal are their mirrors'
        const bool skip = k.col >= p.cols || (KIND >= kApply ? k.row >= p.rows : (k.col >> 7) < (t.row0 >> 7));
        if (!skip) chunk_in<KIND>(tbase + k.tcol, k.half, lane, ws);
        if (ci == kChunks - 1) {   // every column has been read: the accumulator is free
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
        }
        if (!skip) {
          __syncwarp();
          const ChunkIn<KIND> now = in;
          load_next(ci);
          ns_chunk(p, t, k.row, k.col, lane, ws, now, p.diag + static_cast<long long>(t.mat) * p.diag_n);
        } else {
          load_next(ci);
        }
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 1) tmem_dealloc_cg<2>(tmem, 2 * BN);
}

// ---------------------------------------------------- momentum and start

constexpr int kMixThreads = 256;
constexpr int kMixBlocks = 256;   // blocks (and partial sums) per matrix at most

struct MixParams {
  const void* grad;        // matrices [rows, cols], contiguous
  float* momentum;         // or NULL: U = grad
  int grad_f32;
  float mu;
  int nesterov;
  int rows, cols;
  float eps;
  float* partial;          // [matrix][gridDim.x]
  uint32_t* lost;          // cleared here for the products that follow
  __half* hi;
  __half* lo;
  long long pitch, mat;    // stored X
};

// N values of the gradient from element i (N = 8: 16-byte aligned).
template <int N>
__device__ __forceinline__ void grad_at(const MixParams& p, long long i, float (&v)[N]) {
  if constexpr (N == 8) {
    if (p.grad_f32) {
      const float4* q = reinterpret_cast<const float4*>(static_cast<const float*>(p.grad) + i);
      const float4 a = __ldg(q), b = __ldg(q + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.grad) + i));
      v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
      v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    }
  } else {
    v[0] = p.grad_f32 ? static_cast<const float*>(p.grad)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p.grad)[i]);
  }
}
template <int N>
__device__ __forceinline__ void momentum_at(const float* p, float (&v)[N]) {
  if constexpr (N == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *p;
  }
}

// M <- mu M + G and the squares of U = G + mu M (or M), M: there is a
// momentum; one partial sum a block over its share of the matrix's elements, N
// at a time, a few of them in flight.
template <int N, bool M>
__global__ void __launch_bounds__(kMixThreads) muon_mix_kernel(const MixParams p) {
  constexpr int kBatch = M ? 2 : 4;
  __shared__ float red[kMixThreads / 32];
  const long long elems = static_cast<long long>(p.rows) * p.cols, base = blockIdx.y * elems;
  const long long hop = static_cast<long long>(gridDim.x) * kMixThreads * N;
  if ((blockIdx.x | blockIdx.y | threadIdx.x) == 0) *p.lost = 0;
  float s = 0.0f;
  for (long long i0 = (static_cast<long long>(blockIdx.x) * kMixThreads + threadIdx.x) * N; i0 < elems; i0 += kBatch * hop) {
    float u[kBatch][N], m[M ? kBatch : 1][N];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const long long i = i0 + k * hop;
#pragma unroll
      for (int j = 0; j < N; ++j) u[k][j] = 0.0f;
      if (i < elems) {
        grad_at<N>(p, base + i, u[k]);
        if constexpr (M) momentum_at<N>(p.momentum + base + i, m[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      if constexpr (M) {
        const long long i = i0 + k * hop;
        if (i >= elems) continue;
#pragma unroll
        for (int j = 0; j < N; ++j) {
          m[k][j] = fmaf(p.mu, m[k][j], u[k][j]);
          u[k][j] = p.nesterov ? fmaf(p.mu, m[k][j], u[k][j]) : m[k][j];
        }
        float* o = p.momentum + base + i;
        if constexpr (N == 8) {
          reinterpret_cast<float4*>(o)[0] = make_float4(m[k][0], m[k][1], m[k][2], m[k][3]);
          reinterpret_cast<float4*>(o)[1] = make_float4(m[k][4], m[k][5], m[k][6], m[k][7]);
        } else {
          *o = m[k][0];
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j) s = fmaf(u[k][j], u[k][j], s);
    }
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  if (threadIdx.x == 0) {
    for (int w = 1; w < kMixThreads / 32; ++w) s += red[w];
    p.partial[static_cast<long long>(blockIdx.y) * gridDim.x + blockIdx.x] = s;
  }
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}

// X = U / (|U| + eps) as stored halves, zeros in the row padding, 8 columns a
// thread.  N = 8: cols % 8 == 0; N = 1: rows start anywhere, values are read
// one by one (3 x 1000 x 1531: 10 us; a single column a thread 19).
template <int N>
__global__ void __launch_bounds__(kMixThreads) muon_start_kernel(const MixParams p, int parts) {
  __shared__ float red[kMixThreads / 32];
  after_previous();
  const float* part = p.partial + static_cast<long long>(blockIdx.y) * parts;
  float s = threadIdx.x < parts ? part[threadIdx.x] : 0.0f;   // parts <= kMixThreads
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, o);
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = s;
  __syncthreads();
  s = ((red[0] + red[1]) + (red[2] + red[3])) + ((red[4] + red[5]) + (red[6] + red[7]));
  float f = kSx / (sqrtf(s) + p.eps);
  if (f > 3.4e38f) f = 3.4e38f;   // so that zeros stay zeros at any eps (a NaN stays one)
  const long long base = static_cast<long long>(blockIdx.y) * p.rows * p.cols;
  const int groups = static_cast<int>(p.pitch / 8);
  // (row, group) pairs of the matrix, dealt to all its threads
  const long long all = static_cast<long long>(p.rows) * groups;
#pragma unroll 2
  for (long long k = static_cast<long long>(blockIdx.x) * kMixThreads + threadIdx.x; k < all;
       k += static_cast<long long>(gridDim.x) * kMixThreads) {
    const int r = static_cast<int>(k / groups), c = static_cast<int>(k - static_cast<long long>(r) * groups) * 8;
    const long long at = base + static_cast<long long>(r) * p.cols + c, out = blockIdx.y * p.mat + r * p.pitch + c;
    float u[8];
    if (c >= p.cols) {
#pragma unroll
      for (int j = 0; j < 8; ++j) u[j] = 0.0f;
    } else if constexpr (N == 8) {
      grad_at<8>(p, at, u);
      if (p.momentum) {
        float m[8];
        momentum_at<8>(p.momentum + at, m);
#pragma unroll
        for (int j = 0; j < 8; ++j) u[j] = p.nesterov ? fmaf(p.mu, m[j], u[j]) : m[j];
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        u[j] = 0.0f;
        if (c + j < p.cols) {
          grad_at<1>(p, at + j, reinterpret_cast<float(&)[1]>(u[j]));
          if (p.momentum) u[j] = p.nesterov ? fmaf(p.mu, p.momentum[at + j], u[j]) : p.momentum[at + j];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < 8; ++j) u[j] *= f;
    store_hi_lo(p.hi + out, p.lo + out, u);
  }
}

// ------------------------------------------------------------------- host

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

// Smaller sizes at or below this have their apply product read lo as well:
// averaging hi's rounding over few terms leaves more of it (8 x 512 x 256:
// error 1.5e-3 without, 6e-4 with; 120 and 124 us on the tiled kernels).  At
// 1000 x 1531 the result is within 1e-3 without, and lo costs 9 %.
constexpr int kSplitMax = 256;

struct NsLayout {
  int m, k;                    // smaller, larger size
  bool tall, split;
  long long pitch_x, mat_x;    // stored X
  long long pitch_a, mat_a;    // stored A, B
  size_t per_matrix;           // workspace bytes
};

size_t up(size_t v, size_t a) { return (v + a - 1) / a * a; }

NsLayout ns_layout(const moe_muon_config* c) {
  NsLayout L;
  L.tall = c->rows > c->cols;
  L.m = L.tall ? c->cols : c->rows;
  L.k = L.tall ? c->rows : c->cols;
  L.split = L.m <= kSplitMax;
  L.pitch_x = static_cast<long long>(up(c->cols, 64));
  L.mat_x = L.pitch_x * c->rows;
  L.pitch_a = static_cast<long long>(up(L.m, 64));
  L.mat_a = L.pitch_a * L.m;
  const size_t x = static_cast<size_t>(L.mat_x) * 2, a = static_cast<size_t>(L.mat_a) * 2;
  L.per_matrix = (L.split ? 4 : 3) * x + 2 * a + up(L.m * sizeof(float), 16) + kMixBlocks * sizeof(float);
  return L;
}

// Whether the steps keep every matrix's X, A and B within their formats: the
// singular values start in [0, 1] (1 for a matrix of rank one), X's and A's
// elements are at most s and s^2, and B's off its diagonal half the spread of
// b s^2 + c s^4.  The limits leave 6 % to FP16's, and each step's range half a
// percent for rounding: hi and A move A by 3 x 2^-12, X by that times b s^2 +
// 2 c s^4, 0.4 % at the end of steep steps.
bool schedule_in_range(const moe_muon_config* c) {
  double top = 1.0;   // largest singular value before the step
  for (int s = 0; s < c->steps; ++s) {
    const double a = c->coefficients[s][0], b = c->coefficients[s][1], q = c->coefficients[s][2], t = top * top;
    if (!(top <= 15.0 && t <= 120.0)) return false;
    const double peak = q != 0.0 ? -b / (2.0 * q) : 0.0;   // of b t + c t^2
    const double end = (b + q * t) * t, turn = peak > 0.0 && peak < t ? (b + q * peak) * peak : 0.0;
    if (!(std::max({0.0, end, turn}) - std::min({0.0, end, turn}) <= 240.0)) return false;
    auto value = [&](double x2) { return std::fabs((a + (b + q * x2) * x2) * std::sqrt(x2)); };
    double most = value(t);
    // turning points: a + 3 b x^2 + 5 c x^4 = 0
    const double d = 9.0 * b * b - 20.0 * a * q;
    if (q != 0.0 && d >= 0.0) {
      for (double sign : {-1.0, 1.0}) {
        const double x2 = (-3.0 * b + sign * std::sqrt(d)) / (10.0 * q);
        if (x2 > 0.0 && x2 < t) most = std::max(most, value(x2));
      }
    } else if (q == 0.0 && b != 0.0) {
      const double x2 = -a / (3.0 * b);
      if (x2 > 0.0 && x2 < t) most = std::max(most, value(x2));
    }
    if (!std::isfinite(most)) return false;
    top = 1.005 * most;
  }
  return true;
}

bool muon_config_ok(const moe_muon_config* c) {
  if (!c || c->batch < 0 || c->rows < 1 || c->cols < 1) return false;
  if (c->steps < 1 || c->steps > kMaxSteps) return false;
  if (!(c->eps > 0.0f) || c->eps > 3.0e38f) return false;
  bool small = true;
  for (int s = 0; s < c->steps; ++s)
    for (int j = 0; j < 3; ++j) small = small && c->coefficients[s][j] >= -16.0f && c->coefficients[s][j] <= 16.0f;
  return small || schedule_in_range(c);
}

// A CTA pair's matrix sizes: box coordinates and chunk counts are ints.
bool muon_size_ok(const moe_muon_config* c) { return c->rows <= 65536 && c->cols <= 65536; }

// Boxes of two (MN-major B of narrow tiles: one) 64-column chunks of `box_rows` rows.
bool map_of(CUtensorMap* tm, const void* base, long long pitch, int rows, int mats, int box_rows, int chunks) {
  const cuuint64_t d[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(pitch / 64),
                           static_cast<cuuint64_t>(mats)};
  const cuuint64_t st[3] = {static_cast<cuuint64_t>(pitch) * 2, 128, static_cast<cuuint64_t>(pitch) * rows * 2};
  const cuuint32_t bx[4] = {64, static_cast<cuuint32_t>(box_rows), static_cast<cuuint32_t>(chunks), 1};
  return make_tmap_nd(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, d, st, bx, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int KIND, int BN>
cudaError_t launch_ns(const CUtensorMap& a, const CUtensorMap& b, const CUtensorMap& lo, const NsParams& p, int sms,
                      cudaStream_t stream) {
  static PerDeviceOnce once;
  const void* kernel = reinterpret_cast<const void*>(ns_kernel<KIND, BN>);
  cudaError_t e = once.once(
      [&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, NsCfg<BN>::kSmem); });
  if (e != cudaSuccess) return e;
  void* args[4] = {const_cast<CUtensorMap*>(&a), const_cast<CUtensorMap*>(&b), const_cast<CUtensorMap*>(&lo),
                   const_cast<NsParams*>(&p)};
  return launch_dependent(kernel, dim3(2 * std::min(sms / 2, p.total)), kThreads, NsCfg<BN>::kSmem, stream, args);
}

// Tiles of a product: 256 columns wide, or 128 where the pairs get through
// those in less time.  A 128-column tile costs about 0.6 of a 256-column one
// (its operands are three quarters of the other's).  All steps, 256 / 128 columns
// throughout: 3 x 1000 x 1531 265 / 227 us, 2 x 1408 x 2048 324 / 279, 2048 x
// 2048 311 / 281 (rule: 266), 2048 x 7168 561 / 590 (rule: 516), 4096 x 4096
// 1027 / 1407.
template <int KIND>
cudaError_t launch_tiles(const CUtensorMap& a, const CUtensorMap (&b)[2], const CUtensorMap (&lo)[2], NsParams p, int mats,
                         int out_rows, int out_cols, int sms, cudaStream_t stream) {
  constexpr bool sym = KIND == kGram || KIND == kPoly;
  p.valid_cols = out_cols;
  auto count = [&](int bn) {
    p.col_tiles = (out_cols + bn - 1) / bn;
    const int q = (out_rows + 255) / 256, per = 256 / bn;
    p.tiles = q * p.col_tiles - (sym ? per * (q * (q - 1) / 2) : 0);
    p.total = p.tiles * mats;
  };
  auto rounds = [&](int bn) {
    count(bn);
    return (p.total + sms / 2 - 1) / (sms / 2);
  };
  if (0.6f * rounds(128) < rounds(256)) {
    count(128);
    return launch_ns<KIND, 128>(a, b[1], lo[1], p, sms, stream);
  }
  return launch_ns<KIND, 256>(a, b[0], lo[0], p, sms, stream);
}

// What the last product writes and the first kernels read.
struct MuonIo {
  const void* grad;
  int grad_f32;
  float* momentum;
  float mu;
  int nesterov;
  __nv_bfloat16* o16;
  void* weight;
  int weight_f32;
  __nv_bfloat16* w16;
  float decay, rate;
};

// moe_test_muon_lost: the product after which a run's word is set from the host.
std::atomic<int> g_test_lost{-1};

bool test_lost(int product, uint32_t* lost, cudaStream_t stream) {
  if (product != g_test_lost.load(std::memory_order_relaxed)) return true;
  return cudaMemsetAsync(lost, kErrTimeout, 1, stream) == cudaSuccess;
}

moe_status run_muon(const moe_muon_config* c, const MuonIo& io, void* workspace, size_t bytes, uint32_t* err,
                    cudaStream_t stream) {
  const NsLayout L = ns_layout(c);
  const size_t slack = 16 * 256;
  if (bytes < slack + L.per_matrix) return MOE_ERR_CAPACITY;
  int chunk = static_cast<int>(std::min<size_t>((bytes - slack) / L.per_matrix, static_cast<size_t>(c->batch)));
  if (chunk > 65535) chunk = 65535;
  const int sms = device_sms();
  if (sms < 2) return MOE_ERR_CUDA;
  uint8_t* w = static_cast<uint8_t*>(workspace);
  auto take = [&](size_t n) {
    uint8_t* q = w;
    w += up(n, 256);
    return q;
  };
  const size_t nx = static_cast<size_t>(L.mat_x) * 2 * chunk, na = static_cast<size_t>(L.mat_a) * 2 * chunk;
  __half* hi[2] = {reinterpret_cast<__half*>(take(nx)), reinterpret_cast<__half*>(take(nx))};
  __half* lo[2] = {reinterpret_cast<__half*>(take(nx)), nullptr};
  lo[1] = L.split ? reinterpret_cast<__half*>(take(nx)) : lo[0];
  __half* A = reinterpret_cast<__half*>(take(na));
  __half* B = reinterpret_cast<__half*>(take(na));
  float* diag = reinterpret_cast<float*>(take(sizeof(float) * L.m * chunk));
  float* partial = reinterpret_cast<float*>(take(sizeof(float) * kMixBlocks * chunk));
  uint32_t* lost = reinterpret_cast<uint32_t*>(take(sizeof(uint32_t)));

  // tensor maps of X (both buffers), A and B: as the A operand, and as the B
  // operand of 256- and 128-column tiles (B's rows, or X's columns if wide)
  CUtensorMap xa[2], xb[2][2], aa, ab[2], ba, bb[2];
  bool ok = map_of(&aa, A, L.pitch_a, L.m, chunk, 128, 2) && map_of(&ba, B, L.pitch_a, L.m, chunk, 128, 2);
  for (int i = 0; i < 2; ++i) {
    ok = ok && map_of(&xa[i], hi[i], L.pitch_x, c->rows, chunk, 128, 2);
    for (int n = 0; n < 2; ++n) {
      // K-major: BN / 2 rows; MN-major: 128 contraction rows of BN / 2 columns
      ok = ok && map_of(&xb[i][n], hi[i], L.pitch_x, c->rows, chunk, 128, 2 - n);
    }
    ok = ok && map_of(&ab[i], A, L.pitch_a, L.m, chunk, 128 >> i, 2) && map_of(&bb[i], B, L.pitch_a, L.m, chunk, 128 >> i, 2);
  }
  CUtensorMap xl[2][2];   // X's lo half as the operand X is in the apply product
  for (int i = 0; i < 2; ++i)
    for (int n = 0; n < 2; ++n) ok = ok && map_of(&xl[i][n], lo[i], L.pitch_x, c->rows, chunk, 128, L.tall ? 2 : 2 - n);
  CUtensorMap xs[2];      // the same for the small kernel
  for (int i = 0; i < 2; ++i) ok = ok && map_of(&xs[i], lo[i], L.pitch_x, c->rows, chunk, 128, 2);
  CUtensorMap xk[2][2];   // wide: X as the K-major B operand of its own Gram matrix
  for (int i = 0; i < 2; ++i)
    for (int n = 0; n < 2; ++n) ok = ok && map_of(&xk[i][n], hi[i], L.pitch_x, c->rows, chunk, 128 >> n, 2);
  if (!ok) return MOE_ERR_CUDA;

  const long long elems = static_cast<long long>(c->rows) * c->cols;
  for (long long e0 = 0; e0 < c->batch; e0 += chunk) {
    const int n = static_cast<int>(std::min<long long>(chunk, c->batch - e0));
    const long long u0 = e0 * elems;
    MixParams mp{};
    mp.grad = static_cast<const uint8_t*>(io.grad) + u0 * (io.grad_f32 ? 4 : 2);
    mp.momentum = io.momentum ? io.momentum + u0 : nullptr;
    mp.grad_f32 = io.grad_f32;
    mp.mu = io.mu;
    mp.nesterov = io.nesterov;
    mp.rows = c->rows;
    mp.cols = c->cols;
    mp.eps = c->eps;
    mp.partial = partial;
    mp.lost = lost;
    mp.hi = hi[0];
    mp.lo = lo[0];
    mp.pitch = L.pitch_x;
    mp.mat = L.mat_x;
    const bool vec = elems % 8 == 0, vec_rows = c->cols % 8 == 0;
    const int parts = static_cast<int>(std::min<long long>(kMixBlocks, (elems + 8 * kMixThreads - 1) / (8 * kMixThreads)));
    const dim3 mgrid(parts, n);
    if (vec && mp.momentum) muon_mix_kernel<8, true><<<mgrid, kMixThreads, 0, stream>>>(mp);
    else if (vec) muon_mix_kernel<8, false><<<mgrid, kMixThreads, 0, stream>>>(mp);
    else if (mp.momentum) muon_mix_kernel<1, true><<<mgrid, kMixThreads, 0, stream>>>(mp);
    else muon_mix_kernel<1, false><<<mgrid, kMixThreads, 0, stream>>>(mp);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    int parts_arg = parts;
    void* sargs[2] = {&mp, &parts_arg};
    const long long pieces = L.mat_x / 8;
    const dim3 sgrid(static_cast<unsigned>(std::min<long long>(1024, (pieces + kMixThreads - 1) / kMixThreads)), n);
    if (launch_dependent(vec_rows ? reinterpret_cast<const void*>(muon_start_kernel<8>) : reinterpret_cast<const void*>(muon_start_kernel<1>),
                    sgrid, kMixThreads, 0, stream, sargs) != cudaSuccess)
      return MOE_ERR_CUDA;

    const int pairs = L.split ? muon_small_pairs(n, L.m, L.k) : 0;
    if (pairs > 0) {
      SmallParams q{};
      q.mats = n;
      q.pairs = pairs;
      q.steps = c->steps;
      q.tall = L.tall;
      q.kst_gram = (L.k + 127) / 128;
      q.kst_m = (L.m + 127) / 128;
      q.tiles = (L.k + 255) / 256;
      q.m = L.m;
      q.rows = c->rows;
      q.cols = c->cols;
      q.pitch = L.pitch_x;
      q.mat = L.mat_x;
      SmallMaps maps;
      for (int i = 0; i < 2; ++i) {
        q.hi[i] = hi[i];
        q.lo[i] = lo[i];
        maps.x[i] = xa[i];
        maps.lo[i] = xs[i];
      }
      for (int s = 0; s < c->steps; ++s)
        for (int j = 0; j < 3; ++j) q.coef[s][j] = c->coefficients[s][j];
      q.o16 = io.o16 ? io.o16 + u0 : nullptr;
      q.weight = io.weight ? static_cast<uint8_t*>(io.weight) + u0 * (io.weight_f32 ? 4 : 2) : nullptr;
      q.w16 = io.w16 ? io.w16 + u0 : nullptr;
      q.weight_f32 = io.weight_f32;
      q.decay = io.decay;
      q.rate = io.rate;
      q.err = err;
      if (launch_muon_small(maps, q, stream) != cudaSuccess) return MOE_ERR_CUDA;
      continue;
    }
    for (int s = 0; s < c->steps; ++s) {
      const int cur = s & 1;
      const float* co = c->coefficients[s];
      NsParams p{};
      p.err = lost;
      p.rows = L.m;
      p.cols = static_cast<int>(L.pitch_a);
      p.pitch = L.pitch_a;
      p.mat = L.mat_a;
      p.diag = diag;
      p.diag_n = L.m;
      p.a = co[0];
      p.b = co[1];
      p.c = co[2];
      p.a_mn = p.b_mn = L.tall;
      p.kstages = (L.k + 127) / 128;
      p.out_hi = A;
      if (launch_tiles<kGram>(xa[cur], L.tall ? xb[cur] : xk[cur], xl[cur], p, n, L.m, L.m, sms, stream) != cudaSuccess)
        return MOE_ERR_CUDA;
      if (!test_lost(3 * s, lost, stream)) return MOE_ERR_CUDA;
      p.a_mn = p.b_mn = 0;
      p.kstages = (L.m + 127) / 128;
      p.in_hi = A;
      p.out_hi = B;
      if (launch_tiles<kPoly>(aa, ab, xl[cur], p, n, L.m, L.m, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
      if (!test_lost(3 * s + 1, lost, stream)) return MOE_ERR_CUDA;
      p.rows = c->rows;
      p.cols = static_cast<int>(L.pitch_x);
      p.pitch = L.pitch_x;
      p.mat = L.mat_x;
      p.in_hi = hi[cur];
      p.out_hi = hi[cur ^ 1];
      p.in_lo = lo[cur];
      p.out_lo = lo[cur ^ 1];
      p.split = L.split;
      p.diag_cols = L.tall;
      p.b_mn = !L.tall;
      const CUtensorMap& opa = L.tall ? xa[cur] : ba;
      const CUtensorMap (&opb)[2] = L.tall ? bb : xb[cur];
      if (s + 1 < c->steps) {
        if (launch_tiles<kApply>(opa, opb, xl[cur], p, n, c->rows, c->cols, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
        if (!test_lost(3 * s + 2, lost, stream)) return MOE_ERR_CUDA;
      } else {
        p.err = err;
        p.lost = lost;
        p.ucols = c->cols;
        if (io.o16) p.o16 = io.o16 + u0;
        else p.weight = static_cast<uint8_t*>(io.weight) + u0 * (io.weight_f32 ? 4 : 2);
        p.weight_f32 = io.weight_f32;
        p.w16 = io.w16 ? io.w16 + u0 : nullptr;
        p.decay = io.decay;
        p.rate = io.rate;
        const cudaError_t e = io.o16 ? launch_tiles<kFinal>(opa, opb, xl[cur], p, n, c->rows, c->cols, sms, stream)
                                     : launch_tiles<kUpdate>(opa, opb, xl[cur], p, n, c->rows, c->cols, sms, stream);
        if (e != cudaSuccess) return MOE_ERR_CUDA;
      }
    }
  }
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_muon_error_word(uint32_t** device_error_word) {
  if (!device_error_word) return MOE_ERR_INVALID_ARG;
  return cudaGetSymbolAddress(reinterpret_cast<void**>(device_error_word), g_error_word) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_muon_get_error(uint32_t* bits) {
  if (!bits) return MOE_ERR_INVALID_ARG;
  const uint32_t none = 0;
  const bool ok = cudaDeviceSynchronize() == cudaSuccess && cudaMemcpyFromSymbol(bits, g_error_word, sizeof none) == cudaSuccess &&
                  cudaMemcpyToSymbol(g_error_word, &none, sizeof none) == cudaSuccess && cudaDeviceSynchronize() == cudaSuccess;
  return ok ? MOE_OK : MOE_ERR_CUDA;
}

moe_status moe_test_muon_lost(int product) {
  g_test_lost.store(product, std::memory_order_relaxed);
  return MOE_OK;
}

size_t moe_muon_workspace_bytes(const moe_muon_config* cfg, int32_t matrices) {
  if (!muon_config_ok(cfg) || !muon_size_ok(cfg)) return 0;
  const size_t n = matrices > 0 ? static_cast<size_t>(matrices) : 1;
  return ns_layout(cfg).per_matrix * n + 16 * 256;
}

moe_status moe_orthogonalize(const moe_muon_config* cfg, const void* x, moe_type x_type, void* out, void* workspace,
                             size_t workspace_bytes, uint32_t* device_error_word, cudaStream_t stream) {
  if (!muon_config_ok(cfg) || (x_type != MOE_TYPE_BF16 && x_type != MOE_TYPE_FP32)) return MOE_ERR_INVALID_ARG;
  if (!muon_size_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (cfg->batch == 0) return MOE_OK;
  if (!x || !out || !workspace || !device_error_word) return MOE_ERR_INVALID_ARG;
  if (!aligned16(x) || !aligned16(out) || (reinterpret_cast<uintptr_t>(workspace) & 255) ||
      (reinterpret_cast<uintptr_t>(device_error_word) & 3))
    return MOE_ERR_INVALID_ARG;
  MuonIo io{};
  io.grad = x;
  io.grad_f32 = x_type == MOE_TYPE_FP32;
  io.o16 = static_cast<__nv_bfloat16*>(out);
  return run_muon(cfg, io, workspace, workspace_bytes, device_error_word, stream);
}

moe_status moe_muon_update(const moe_muon_config* cfg, const moe_muon_rates* rates, void* weight, moe_type weight_type,
                           const void* grad, moe_type grad_type, float* momentum, void* weight_bf16, void* workspace,
                           size_t workspace_bytes, uint32_t* device_error_word, cudaStream_t stream) {
  if (!muon_config_ok(cfg) || !rates) return MOE_ERR_INVALID_ARG;
  if ((weight_type != MOE_TYPE_BF16 && weight_type != MOE_TYPE_FP32) ||
      (grad_type != MOE_TYPE_BF16 && grad_type != MOE_TYPE_FP32))
    return MOE_ERR_INVALID_ARG;
  const float f[4] = {rates->lr, rates->mu, rates->weight_decay, rates->scale};
  for (float v : f)
    if (!(v >= -3.0e38f && v <= 3.0e38f)) return MOE_ERR_INVALID_ARG;
  if (weight_bf16 && weight_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (!muon_size_ok(cfg)) return MOE_ERR_UNSUPPORTED;
  if (cfg->batch == 0) return MOE_OK;
  if (!weight || !grad || !momentum || !workspace || !device_error_word) return MOE_ERR_INVALID_ARG;
  if (!aligned16(weight) || !aligned16(grad) || !aligned16(momentum) || !aligned16(weight_bf16) ||
      (reinterpret_cast<uintptr_t>(workspace) & 255) || (reinterpret_cast<uintptr_t>(device_error_word) & 3))
    return MOE_ERR_INVALID_ARG;
  MuonIo io{};
  io.grad = grad;
  io.grad_f32 = grad_type == MOE_TYPE_FP32;
  io.momentum = momentum;
  io.mu = rates->mu;
  io.nesterov = rates->nesterov != 0;
  io.weight = weight;
  io.weight_f32 = weight_type == MOE_TYPE_FP32;
  io.w16 = static_cast<__nv_bfloat16*>(weight_bf16);
  io.decay = static_cast<float>(1.0 - static_cast<double>(rates->lr) * rates->weight_decay);
  io.rate = static_cast<float>(static_cast<double>(rates->lr) * rates->scale);
  return run_muon(cfg, io, workspace, workspace_bytes, device_error_word, stream);
}

}  // extern "C"
