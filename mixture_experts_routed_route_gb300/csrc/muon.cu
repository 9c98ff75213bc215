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
// X is stored times 2^12, A and B times 2^11 (exact powers of two), so that
// FP16 keeps its 11 bits down to elements of 1.5e-8 of X, and B's
// off-diagonal elements (below 32 for |coefficients| of this kind of
// polynomial) stay in range.
//
// Each product is one persistent launch over 256 x 256 output tiles of all
// matrices, a tile on a CTA pair (cta_group::2, M = 256, N = 256: per SM a
// stage of 128 contraction elements is 64 KB of operands for 2 x 256 x 256 x
// 128 flops on the pair).  A and B are symmetric: only tiles on or above
// the diagonal are computed, and their epilogue stores the mirror image too.
// Tall and wide matrices need no transposes: the operand whose contraction
// index is not the fastest one in memory is read MN-major by the same tensor
// map (64-column chunks as an axis of their own).
//
// Warp roles: warp 0 TMA producer, warp 1 TMEM allocation and (rank 0) MMA
// issue for the pair, warps 2 .. 9 epilogue (lane quadrant w % 4, columns
// 128 h .. 128 h + 127 of the tile).  Both CTAs' loads complete on rank 0's
// barrier of the stage.
#include <cuda_fp16.h>

#include <algorithm>

#include "kernels.cuh"
#include "moe_gb300.h"

namespace moe {

namespace {

constexpr float kSx = 4096.0f;   // stored X = X * kSx
constexpr float kSb = 2048.0f;   // stored A, B = A, B * kSb
constexpr int kBoxBytes = 2 * 128 * 128;   // two 64-element chunks of 128 rows
constexpr int kStageBytes = 2 * kBoxBytes;
constexpr int kStages = 3;
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kSmem = 1024 + kStages * kStageBytes + 256;
constexpr int kMaxSteps = MOE_MUON_MAX_STEPS;

enum NsKind { kGram, kPoly, kApply, kFinal };

struct NsParams {
  int tiles;            // per matrix
  int total;            // tiles of all matrices
  int n256;             // 256-row blocks of a symmetric output
  int col_tiles;        // 256-column tiles of an apply output
  int kstages;          // stages of 128 contraction elements
  int a_mn, b_mn;       // operand read MN-major
  int rows, cols;       // valid rows, columns written (a multiple of 8)
  long long pitch;      // elements per stored row (multiple of 64)
  long long mat;        // elements per stored matrix
  const __half* in_hi;  // poly: A; apply: X hi
  __half* out_hi;       // gram: A; poly: B; apply: X hi (next)
  __half* lo;           // apply: X lo, in place
  float* diag;          // [matrix][diag_n]: B's diagonal
  int diag_n;
  int diag_cols;        // apply: the diagonal scales columns (tall) or rows (wide)
  float a, b, c;
  // final step: the caller's tensors [rows, ucols] of matrix `first` on
  __nv_bfloat16* o16;   // orthogonalised update
  void* weight;         // or the weight, in place
  __nv_bfloat16* w16;   // and its BF16 copy
  int weight_f32;
  int ucols;
  float decay, rate;    // W <- decay W - rate X
  uint32_t* err;
};

// Both CTAs' loads of a stage complete on rank 0's barrier (the address of
// an mbarrier in rank 0, for either CTA of the pair).
__device__ __forceinline__ void tma_load_4d_pair(void* smem_dst, const CUtensorMap* tm, uint32_t bar, int x, int y,
                                                 int z, int w) {
  asm volatile(
      "cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5, %6}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(tm)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(w)
      : "memory");
}

// MN-major FP16 tile in the 128-byte swizzle: groups of 64 elements along
// M (or N), each 128 rows (contraction elements) of 128 bytes; 8-row atoms
// 1024 bytes apart along the contraction, groups 16 KB apart.
__device__ __forceinline__ uint64_t sdesc_mn_f16(uint32_t saddr) {
  uint64_t d = 0;
  d |= static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4);
  d |= static_cast<uint64_t>(16384 >> 4) << 16;
  d |= static_cast<uint64_t>(1024 >> 4) << 32;
  d |= static_cast<uint64_t>(1) << 46;
  d |= static_cast<uint64_t>(2) << 61;
  return d;
}

struct NsTile {
  int mat, row0, col0;   // this CTA's 128 output rows, the pair's 256 columns
};

// Symmetric outputs: tile t of the upper triangle of n256 x n256 blocks.
template <int KIND>
__device__ __forceinline__ NsTile ns_tile(const NsParams& p, int tile, int rank) {
  NsTile t;
  t.mat = tile / p.tiles;
  int i = tile - t.mat * p.tiles, q = 0;
  if (KIND == kGram || KIND == kPoly) {
    for (; i >= p.n256 - q; ++q) i -= p.n256 - q;
    t.row0 = q * 256 + 128 * rank;
    t.col0 = (q + i) * 256;
  } else {
    q = i / p.col_tiles;
    t.row0 = q * 256 + 128 * rank;
    t.col0 = (i - q * p.col_tiles) * 256;
  }
  return t;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
  const __half2 v = __floats2half2_rn(lo, hi);
  return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ float half_lo(uint32_t u) { return __half2float(__ushort_as_half(static_cast<unsigned short>(u & 0xFFFFu))); }
__device__ __forceinline__ float half_hi(uint32_t u) { return __half2float(__ushort_as_half(static_cast<unsigned short>(u >> 16))); }

// One row's 8 columns of hi + lo halves from FP32 values (stored scale).
__device__ __forceinline__ void store_hi_lo(__half* hi, __half* lo, const float* v) {
  uint32_t h[4], l[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    h[j] = pack_half2(v[2 * j], v[2 * j + 1]);
    l[j] = pack_half2(v[2 * j] - half_lo(h[j]), v[2 * j + 1] - half_hi(h[j]));
  }
  *reinterpret_cast<uint4*>(hi) = make_uint4(h[0], h[1], h[2], h[3]);
  *reinterpret_cast<uint4*>(lo) = make_uint4(l[0], l[1], l[2], l[3]);
}

// 32 columns of row r (this lane) and its columns c .. c + 31, from the
// accumulator values v.
template <int KIND>
__device__ __forceinline__ void ns_chunk(const NsParams& p, const NsTile& t, int r, int c, const uint32_t (&v)[32]) {
  const bool in_rows = r < p.rows;
  const long long at = t.mat * p.mat + static_cast<long long>(r) * p.pitch + c;
  if constexpr (KIND == kGram || KIND == kPoly) {
    uint32_t w[16];
    if constexpr (KIND == kGram) {
#pragma unroll
      for (int j = 0; j < 16; ++j)
        w[j] = pack_half2(__uint_as_float(v[2 * j]) * (kSb / (kSx * kSx)), __uint_as_float(v[2 * j + 1]) * (kSb / (kSx * kSx)));
    } else {
      const float cs = p.c * (1.0f / kSb);
#pragma unroll
      for (int g = 0; g < 4; ++g) {
        uint4 u = make_uint4(0, 0, 0, 0);
        if (in_rows && c + 8 * g < p.cols) u = *reinterpret_cast<const uint4*>(p.in_hi + at + 8 * g);
        const uint32_t a[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int k = 8 * g + 2 * j;
          float x0 = fmaf(cs, __uint_as_float(v[k]), p.b * half_lo(a[j]));
          float x1 = fmaf(cs, __uint_as_float(v[k + 1]), p.b * half_hi(a[j]));
          if (c + k == r) {
            if (in_rows) p.diag[static_cast<long long>(t.mat) * p.diag_n + r] = x0 * (1.0f / kSb);
            x0 = 0.0f;
          }
          if (c + k + 1 == r) {
            if (in_rows) p.diag[static_cast<long long>(t.mat) * p.diag_n + r] = x1 * (1.0f / kSb);
            x1 = 0.0f;
          }
          w[4 * g + j] = pack_half2(x0, x1);
        }
      }
    }
    if (in_rows) {
#pragma unroll
      for (int g = 0; g < 4; ++g)
        if (c + 8 * g < p.cols)
          *reinterpret_cast<uint4*>(p.out_hi + at + 8 * g) = make_uint4(w[4 * g], w[4 * g + 1], w[4 * g + 2], w[4 * g + 3]);
    }
    // the mirror image of blocks above the diagonal (column r of rows c ..)
    if ((c >> 7) > (r >> 7) && r < p.cols) {
      __half* m = p.out_hi + t.mat * p.mat + r;
#pragma unroll
      for (int k = 0; k < 32; ++k)
        if (c + k < p.rows)
          m[(c + k) * p.pitch] = __ushort_as_half(static_cast<unsigned short>((k & 1) ? (w[k >> 1] >> 16) : (w[k >> 1] & 0xFFFFu)));
    }
  } else {
    if (!in_rows) return;
    const float* d = p.diag + static_cast<long long>(t.mat) * p.diag_n;
    const float drow = p.diag_cols ? 0.0f : d[r];
#pragma unroll
    for (int g = 0; g < 4; ++g) {
      const int cg = c + 8 * g;
      if (cg >= p.cols) continue;
      const uint4 uh = *reinterpret_cast<const uint4*>(p.in_hi + at + 8 * g);
      const uint4 ul = *reinterpret_cast<const uint4*>(p.lo + at + 8 * g);
      const uint32_t h[4] = {uh.x, uh.y, uh.z, uh.w}, l[4] = {ul.x, ul.y, ul.z, ul.w};
      float x[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[2 * j] = half_lo(h[j]) + half_lo(l[j]);
        x[2 * j + 1] = half_hi(h[j]) + half_hi(l[j]);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float dj = p.diag_cols ? (cg + j < p.diag_n ? d[cg + j] : 0.0f) : drow;
        x[j] = fmaf(p.a + dj, x[j], __uint_as_float(v[8 * g + j]) * (1.0f / kSb));
      }
      if constexpr (KIND == kApply) {
        store_hi_lo(p.out_hi + at + 8 * g, p.lo + at + 8 * g, x);
      } else {
        const long long u = (static_cast<long long>(t.mat) * p.rows + r) * p.ucols + cg;
        if (p.o16) {
          if (p.ucols % 8 == 0) {
            *reinterpret_cast<uint4*>(p.o16 + u) =
                make_uint4(pack_bf16x2(x[0] / kSx, x[1] / kSx), pack_bf16x2(x[2] / kSx, x[3] / kSx),
                           pack_bf16x2(x[4] / kSx, x[5] / kSx), pack_bf16x2(x[6] / kSx, x[7] / kSx));
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (cg + j < p.ucols) p.o16[u + j] = __float2bfloat16_rn(x[j] / kSx);
          }
        } else {
          const float rate = p.rate / kSx;
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            if (cg + j >= p.ucols) continue;
            float w;
            if (p.weight_f32) {
              float* q = static_cast<float*>(p.weight) + u + j;
              w = fmaf(p.decay, *q, -rate * x[j]);
              *q = w;
            } else {
              __nv_bfloat16* q = static_cast<__nv_bfloat16*>(p.weight) + u + j;
              w = fmaf(p.decay, __bfloat162float(*q), -rate * x[j]);
              *q = __float2bfloat16_rn(w);
            }
            if (p.w16) p.w16[u + j] = __float2bfloat16_rn(w);
          }
        }
      }
    }
  }
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitTimeoutCycles / 8) return;
  }
}

template <int KIND>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kThreads, 1)
    ns_kernel(const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB, const NsParams p) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint64_t* full = reinterpret_cast<uint64_t*>(smem + kStages * kStageBytes);   // rank 0: both CTAs' operands landed
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
    tmem_alloc_cg<2>(tmem_slot, 512);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  cluster_sync();   // the other CTA's barriers exist before anything arrives on them

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    uint32_t it = 0;
    bool ok = true;
    for (int tile = cid; ok && tile < p.total; tile += ncl) {
      const NsTile t = ns_tile<KIND>(p, tile, rank);
      const int brow = t.col0 + 128 * rank;   // this CTA's half of the N rows
      for (int ks = 0; ks < p.kstages; ++ks, ++it) {
        const uint32_t slot = it % kStages, ph = (it / kStages) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&empty[slot], ph ^ 1, abort_flag, p.err))) {
          ok = false;
          break;
        }
        if (lane == 0) {
          uint8_t* sa = smem + slot * kStageBytes;
          const uint32_t bar = cluster_addr(&full[slot], 0);
          if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * kStageBytes);
          const int k0 = ks * 128;
          if (p.a_mn) tma_load_4d_pair(sa, &tmA, bar, 0, k0, t.row0 >> 6, t.mat);
          else tma_load_4d_pair(sa, &tmA, bar, 0, t.row0, k0 >> 6, t.mat);
          if (p.b_mn) tma_load_4d_pair(sa + kBoxBytes, &tmB, bar, 0, k0, brow >> 6, t.mat);
          else tma_load_4d_pair(sa + kBoxBytes, &tmB, bar, 0, brow, k0 >> 6, t.mat);
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
      const uint32_t idesc = (1u << 4) | ((256u >> 3) << 17) | ((256u >> 4) << 24) | (p.a_mn ? kIdescAMnMajor : 0u) |
                             (p.b_mn ? (1u << 16) : 0u);
      uint32_t it = 0, tc = 0;
      bool ok = true;
      for (int tile = cid; ok && tile < p.total; tile += ncl, ++tc) {
        const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
        if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&tempty[acc], aph ^ 1, abort_flag, p.err))) break;
        tc_fence_after();
        const uint32_t d_tmem = tmem + acc * 256;
        for (int ks = 0; ks < p.kstages; ++ks, ++it) {
          const uint32_t slot = it % kStages, ph = (it / kStages) & 1;
          if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&full[slot], ph, abort_flag, p.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          if (lane == 0) {
            const uint32_t sa = smem_u32(smem + slot * kStageBytes), sb = sa + kBoxBytes;
#pragma unroll
            for (int j = 0; j < 8; ++j) {   // 16 contraction elements each
              const uint64_t ad = p.a_mn ? sdesc_mn_f16(sa + j * 2048) : sdesc_k_sw128(sa + (j >> 2) * 16384 + (j & 3) * 32);
              const uint64_t bd = p.b_mn ? sdesc_mn_f16(sb + j * 2048) : sdesc_k_sw128(sb + (j >> 2) * 16384 + (j & 3) * 32);
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
      if (lane == 0) {
        tc_commit_pair(drain);
        drain_wait(drain, 0);
      }
      __syncwarp();
    }
  } else {
    // --------------------------------------------------------- epilogue
    const int q = warp & 3, h = (warp - 2) >> 2;
    const uint32_t tempty0 = cluster_addr(tempty, 0);
    uint32_t tc = 0;
    for (int tile = cid; tile < p.total; tile += ncl, ++tc) {
      const NsTile t = ns_tile<KIND>(p, tile, rank);
      const uint32_t acc = tc & 1, aph = (tc >> 1) & 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&tfull[acc], aph, abort_flag, p.err))) break;
      tc_fence_after();
      const uint32_t tbase = tmem + acc * 256 + (static_cast<uint32_t>(q * 32) << 16) + 128 * h;
      const int r = t.row0 + q * 32 + lane, c = t.col0 + 128 * h;
      // a symmetric tile's block below the diagonal is its mirror's
      const bool skip = (KIND == kGram || KIND == kPoly) && (c >> 7) < (t.row0 >> 7);
#pragma unroll 1
      for (int ci = 0; ci < 4; ++ci) {
        if (skip || c + 32 * ci >= p.cols) continue;
        uint32_t v[32];
        tmem_ld32(tbase + 32 * ci, v);
        tmem_ld_wait();
        ns_chunk<KIND>(p, t, r, c + 32 * ci, v);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 1) tmem_dealloc_cg<2>(tmem, 512);
}

// ---------------------------------------------------- momentum and start

constexpr int kMixThreads = 256;
constexpr int kMixBlocks = 64;   // blocks (and partial sums) per matrix at most

struct MixParams {
  const void* grad;        // matrices [rows, cols], contiguous
  float* momentum;         // or NULL: U = grad
  int grad_f32;
  float mu;
  int nesterov;
  int rows, cols;
  float eps;
  float* partial;          // [matrix][gridDim.x]
  __half* hi;
  __half* lo;
  long long pitch, mat;    // stored X
};

__device__ __forceinline__ float grad_at(const MixParams& p, long long i) {
  return p.grad_f32 ? static_cast<const float*>(p.grad)[i]
                    : __bfloat162float(static_cast<const __nv_bfloat16*>(p.grad)[i]);
}

__device__ __forceinline__ float update_at(const MixParams& p, long long i, float m) {
  const float g = grad_at(p, i);
  return p.momentum ? (p.nesterov ? fmaf(p.mu, m, g) : m) : g;
}

// M <- mu M + G and the squares of U = G + mu M (or M): one partial sum a
// block, rows dealt to the blocks in turn.
__global__ void __launch_bounds__(kMixThreads) muon_mix_kernel(const MixParams p) {
  __shared__ float red[kMixThreads / 32];
  const long long base = static_cast<long long>(blockIdx.y) * p.rows * p.cols;
  float s = 0.0f;
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const long long row = base + static_cast<long long>(r) * p.cols;
    for (int c = threadIdx.x; c < p.cols; c += kMixThreads) {
      float m = 0.0f;
      if (p.momentum) {
        m = fmaf(p.mu, p.momentum[row + c], grad_at(p, row + c));
        p.momentum[row + c] = m;
      }
      const float u = update_at(p, row + c, m);
      s = fmaf(u, u, s);
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
}

// X = U / (|U| + eps) as stored halves, zeros in the row padding.
__global__ void __launch_bounds__(kMixThreads) muon_start_kernel(const MixParams p, int parts) {
  const float* part = p.partial + static_cast<long long>(blockIdx.y) * parts;
  float s = 0.0f;
  for (int i = 0; i < parts; ++i) s += part[i];
  const float f = kSx / (sqrtf(s) + p.eps);
  const long long base = static_cast<long long>(blockIdx.y) * p.rows * p.cols;
  const int groups = static_cast<int>(p.pitch >> 3);
  for (int r = blockIdx.x; r < p.rows; r += gridDim.x) {
    const long long row = base + static_cast<long long>(r) * p.cols;
    const long long out = blockIdx.y * p.mat + r * p.pitch;
    for (int g = threadIdx.x; g < groups; g += kMixThreads) {
      float v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const int c = 8 * g + j;
        v[j] = c < p.cols ? f * update_at(p, row + c, p.momentum ? p.momentum[row + c] : 0.0f) : 0.0f;
      }
      store_hi_lo(p.hi + out + 8 * g, p.lo + out + 8 * g, v);
    }
  }
}

// ------------------------------------------------------------------- host

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct NsLayout {
  int m, k;                    // smaller, larger size
  bool tall;
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
  L.pitch_x = static_cast<long long>(up(c->cols, 64));
  L.mat_x = L.pitch_x * c->rows;
  L.pitch_a = static_cast<long long>(up(L.m, 64));
  L.mat_a = L.pitch_a * L.m;
  size_t x = static_cast<size_t>(L.mat_x) * 2, a = static_cast<size_t>(L.mat_a) * 2;
  L.per_matrix = 3 * x + 2 * a + up(L.m * sizeof(float), 16) + kMixBlocks * sizeof(float);
  return L;
}

bool muon_config_ok(const moe_muon_config* c) {
  if (!c || c->batch < 0 || c->rows < 1 || c->cols < 1) return false;
  if (c->steps < 1 || c->steps > kMaxSteps) return false;
  if (!(c->eps > 0.0f) || c->eps > 3.0e38f) return false;
  for (int s = 0; s < c->steps; ++s)
    for (int j = 0; j < 3; ++j)
      if (!(c->coefficients[s][j] >= -16.0f && c->coefficients[s][j] <= 16.0f)) return false;
  return true;
}

// A CTA pair's matrix sizes: box coordinates and chunk counts are ints.
bool muon_size_ok(const moe_muon_config* c) { return c->rows <= 65536 && c->cols <= 65536; }

bool map_of(CUtensorMap* tm, const void* base, long long pitch, int rows, int mats) {
  const cuuint64_t d[4] = {64, static_cast<cuuint64_t>(rows), static_cast<cuuint64_t>(pitch / 64),
                           static_cast<cuuint64_t>(mats)};
  const cuuint64_t st[3] = {static_cast<cuuint64_t>(pitch) * 2, 128, static_cast<cuuint64_t>(pitch) * rows * 2};
  const cuuint32_t bx[4] = {64, 128, 2, 1};
  return make_tmap_nd(tm, CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, base, d, st, bx, CU_TENSOR_MAP_SWIZZLE_128B);
}

template <int KIND>
cudaError_t launch_ns(const CUtensorMap& a, const CUtensorMap& b, const NsParams& p, int sms, cudaStream_t stream) {
  static PerDeviceOnce once;
  cudaError_t e = once.once(
      [] { return cudaFuncSetAttribute(ns_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (e != cudaSuccess) return e;
  int pairs = sms / 2;
  if (p.total < pairs) pairs = p.total;
  ns_kernel<KIND><<<2 * pairs, kThreads, kSmem, stream>>>(a, b, p);
  return cudaGetLastError();
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

int device_sms() {
  static PerDeviceOnce once;
  static int sms[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const cudaError_t e = once.once([&] { return cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev); });
  return e == cudaSuccess ? sms[dev] : 0;
}

moe_status run_muon(const moe_muon_config* c, const MuonIo& io, void* workspace, size_t bytes, uint32_t* err,
                    cudaStream_t stream) {
  const NsLayout L = ns_layout(c);
  const size_t slack = 8 * 256;
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
  __half* lo = reinterpret_cast<__half*>(take(nx));
  __half* A = reinterpret_cast<__half*>(take(na));
  __half* B = reinterpret_cast<__half*>(take(na));
  float* diag = reinterpret_cast<float*>(take(sizeof(float) * L.m * chunk));
  float* partial = reinterpret_cast<float*>(take(sizeof(float) * kMixBlocks * chunk));

  CUtensorMap tx[2], ta, tb;
  if (!map_of(&tx[0], hi[0], L.pitch_x, c->rows, chunk) || !map_of(&tx[1], hi[1], L.pitch_x, c->rows, chunk) ||
      !map_of(&ta, A, L.pitch_a, L.m, chunk) || !map_of(&tb, B, L.pitch_a, L.m, chunk))
    return MOE_ERR_CUDA;

  const long long elems = static_cast<long long>(c->rows) * c->cols;
  for (int e0 = 0; e0 < c->batch; e0 += chunk) {
    const int n = std::min(chunk, c->batch - e0);
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
    mp.hi = hi[0];
    mp.lo = lo;
    mp.pitch = L.pitch_x;
    mp.mat = L.mat_x;
    const int parts = std::min(kMixBlocks, c->rows);
    muon_mix_kernel<<<dim3(parts, n), kMixThreads, 0, stream>>>(mp);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
    muon_start_kernel<<<dim3(std::min(c->rows, 1024), n), kMixThreads, 0, stream>>>(mp, parts);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;

    for (int s = 0; s < c->steps; ++s) {
      const int cur = s & 1;
      const float* co = c->coefficients[s];
      NsParams p{};
      p.err = err;
      p.n256 = (L.m + 255) / 256;
      p.tiles = p.n256 * (p.n256 + 1) / 2;
      p.total = p.tiles * n;
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
      if (launch_ns<kGram>(tx[cur], tx[cur], p, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
      p.a_mn = p.b_mn = 0;
      p.kstages = (L.m + 127) / 128;
      p.in_hi = A;
      p.out_hi = B;
      if (launch_ns<kPoly>(ta, ta, p, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
      p.rows = c->rows;
      p.cols = static_cast<int>(L.pitch_x);
      p.pitch = L.pitch_x;
      p.mat = L.mat_x;
      p.col_tiles = (c->cols + 255) / 256;
      p.tiles = (c->rows + 255) / 256 * p.col_tiles;
      p.total = p.tiles * n;
      p.in_hi = hi[cur];
      p.out_hi = hi[cur ^ 1];
      p.lo = lo;
      p.diag_cols = L.tall;
      p.b_mn = !L.tall;
      const CUtensorMap& opa = L.tall ? tx[cur] : tb;
      const CUtensorMap& opb = L.tall ? tb : tx[cur];
      if (s + 1 < c->steps) {
        if (launch_ns<kApply>(opa, opb, p, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
      } else {
        p.ucols = c->cols;
        if (io.o16) p.o16 = io.o16 + u0;
        else p.weight = static_cast<uint8_t*>(io.weight) + u0 * (io.weight_f32 ? 4 : 2);
        p.weight_f32 = io.weight_f32;
        p.w16 = io.w16 ? io.w16 + u0 : nullptr;
        p.decay = io.decay;
        p.rate = io.rate;
        if (launch_ns<kFinal>(opa, opb, p, sms, stream) != cudaSuccess) return MOE_ERR_CUDA;
      }
    }
  }
  return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_muon_workspace_bytes(const moe_muon_config* cfg, int32_t matrices) {
  if (!muon_config_ok(cfg) || !muon_size_ok(cfg)) return 0;
  const size_t n = matrices > 0 ? static_cast<size_t>(matrices) : 1;
  return ns_layout(cfg).per_matrix * n + 8 * 256;
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
