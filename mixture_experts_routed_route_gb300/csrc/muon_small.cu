// Newton-Schulz steps of small matrices (smaller size m at most 256): one to
// four CTA pairs, a cluster, take a matrix through all its steps in one
// launch.
//
// What bounds such matrices is not work but the chain of dependent products:
// as separate launches a step is three of them at about 7 us each, of which
// the tensor cores take a tenth.  Here A and B never leave the chip: each CTA
// of a pair keeps its 128 rows of them (64 KB) in shared memory, in the layout
// in which the next product reads them, as both its A and its half of the B
// operand, A being symmetric.  X still goes through memory (L2), in hi and lo
// halves as in muon.cu, so any k fits.  With several pairs a matrix, each pair
// computes A and B for itself (nothing to exchange, and the products are
// short) and takes every pairs-th tile of 256 rows or columns of the new X.
//
// m x k, this kernel / tiled kernels, five steps and the two kernels before
// them (results are equal bit by bit):
//   8 x 256 x 256   83 / 119 us      64 x 256 x 256   92 / 180 us
//   8 x 256 x 512   90 / 125         64 x 256 x 1024 231 / 369
//   1 x 64 x 256    65 / 82          64 x 256 x 2048 447 / 614
//   8 x 256 x 4096 259 / 271          1 x 256 x 4096 246 / 191  (not taken)
// A step on one tile is about 33000 cycles: loads and the first product 3700,
// A's epilogue 3000, the second product 3000, B's 4200, the diagonal's way to
// both CTAs 1500, the third product (over hi and lo) 4500, X's epilogue 9000
// (X through L2, a cycle of L1 a line, the chunks turned around in shared
// memory) and 1500 until its stores can be seen by the next step's loads.  Sixteen epilogue
// warps: eight took 107 us instead of 96 at 8 x 512 x 256.
//
// Warp roles as in muon.cu.  Hand-overs:
//   full / empty   ring of 32 KB operand boxes, loads of both CTAs complete on
//                  rank 0's barrier; in the Gram product one box serves as
//                  both operands
//   tfull / tempty accumulators (two of 256 columns)
//   ready          rank 0: all 16 epilogue warps stored A (then B) in shared
//                  memory for the tensor core of their own SM
//   dready         all warps of the pair stored their part of B's diagonal in
//                  both CTAs
//   xready         all warps of the cluster stored their part of the new X in
//                  memory, which the next step's loads read; X's two buffers
//                  take turns, and nobody reads the older one after this
// The last three carry data across SMs: release and acquire at cluster scope.
#include <algorithm>

#include "muon_core.cuh"

namespace moe {

namespace {

constexpr int kSlots = 3, kSlotBytes = 2 * 128 * 128;
constexpr int kSmallWarps = 16, kSmallThreads = 32 * (2 + kSmallWarps);   // epilogue warps
constexpr int kRegion = 4 * 128 * 128;   // A or B: 128 rows of 256 columns in 64-column chunks
constexpr int kSmallSmem = 1024 + kSlots * kSlotBytes + kRegion + kSmallWarps * 4096 + 1024 + 256;
static_assert(kSmallSmem <= 232448, "shared memory per CTA");

// Arrive on a barrier of CTA `rank`'s counterpart of `bar`, cluster-scope release.
__device__ __forceinline__ void mbar_arrive_release(uint64_t* bar, uint32_t rank) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(cluster_addr(bar, rank)) : "memory");
}

// mbar_wait with cluster-scope acquire.
__device__ __forceinline__ bool mbar_wait_acquire(uint64_t* bar, uint32_t parity, volatile int* abort_flag, uint32_t* err) {
  const long long t0 = clock64();
  while (true) {
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity), "n"(kClusterWaitNs)
        : "memory");
    if (ok) return true;
    if (*abort_flag) return false;
    if (clock64() - t0 > kWaitTimeoutCycles) {
      *abort_flag = 1;
      atomicOr(err, kErrTimeout);
      return false;
    }
  }
}

__device__ __forceinline__ void st_cluster_f32(float* p, uint32_t rank, float v) {
  asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(cluster_addr(p, rank)), "f"(v) : "memory");
}

// A pair's tiles of the new X through its epilogue warps; KIND as in muon.cu.
// Of a tile, warp (q, h) has rows 32 q .. and columns 64 h .., in two halves of
// the rows; where X has no more than 64 or 128 columns the warps of a quadrant
// share those.
template <int KIND>
__device__ __forceinline__ bool small_apply(const SmallParams& sp, const NsParams& p, int mat, int rank, int pair, int q, int h,
                                            int lane, float* ws, uint64_t* tfull, uint32_t tempty0, uint32_t tmem,
                                            uint32_t& tc, const float* d, volatile int* abort_flag) {
  const int share = !sp.tall || p.cols > 128 ? 2 : p.cols > 64 ? 1 : 0;
  const int tcol = 64 * (h & ((1 << share) - 1)), half0 = h >> share;
  for (int tile = pair; tile < sp.tiles; tile += sp.pairs, ++tc) {
    NsTile t;
    t.mat = mat;
    t.row0 = (sp.tall ? tile * 256 : 0) + 128 * rank;
    t.col0 = sp.tall ? 0 : tile * 256;
    t.n = 256;
    const uint32_t acc = tc & 1, par = (tc >> 1) & 1;
    ChunkIn<KIND, true> in;
    const int r0 = t.row0 + 32 * q + 16 * half0, c0 = t.col0 + tcol;
    load_chunk_in(p, mat, r0, c0, lane, in);
    if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&tfull[acc], par, abort_flag, p.err))) return false;
    tc_fence_after();
    const uint32_t tbase = tmem + acc * 256 + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll 1
    for (int ci = 0; ci < 2; ++ci) {
      const bool skip = c0 >= p.cols || r0 + 16 * ci >= p.rows || half0 + ci > (share == 2 ? 1 : half0 & 1);
      if (!skip && ci > 0) load_chunk_in(p, mat, r0 + 16, c0, lane, in);
      if (!skip) chunk_in<KIND>(tbase + tcol, half0 + ci, lane, ws);
      if (ci == 1) {
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
      }
      if (!skip) {
        __syncwarp();
        ns_chunk(p, t, r0 + 16 * ci, c0, lane, ws, in, d);
      }
    }
  }
  return true;
}

__global__ void __launch_bounds__(kSmallThreads, 1)
    muon_small_kernel(const __grid_constant__ SmallMaps maps, const __grid_constant__ SmallParams sp) {
  extern __shared__ uint8_t smem_raw[];
  uint8_t* ring = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
  uint8_t* region = ring + kSlots * kSlotBytes;
  float* turn = reinterpret_cast<float*>(region + kRegion);
  float* diag = turn + kSmallWarps * 1024;                                // [256]
  uint64_t* full = reinterpret_cast<uint64_t*>(diag + 256);
  uint64_t* empty = full + kSlots;
  uint64_t* tfull = empty + kSlots;
  uint64_t* tempty = tfull + 2;
  uint64_t* ready = tempty + 2;
  uint64_t* dready = ready + 1;
  uint64_t* xready = dready + 1;
  uint64_t* drain = xready + 1;
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
  volatile int* abort_flag = reinterpret_cast<volatile int*>(tmem_slot + 1);

  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int crank = static_cast<int>(cluster_ctarank()), rank = crank & 1, pair = crank >> 1;
  const int ctas = 2 * sp.pairs, lead = 2 * pair;      // of the cluster; rank 0 of this pair
  const uint16_t both = static_cast<uint16_t>(3u << lead);
  const int cid = blockIdx.x / ctas, ncl = gridDim.x / ctas;
  if (threadIdx.x == 0) {
    for (int s = 0; s < kSlots; ++s) {
      mbar_init(&full[s], 1);
      mbar_init(&empty[s], 1);
    }
    for (int a = 0; a < 2; ++a) {
      mbar_init(&tfull[a], 1);
      mbar_init(&tempty[a], 2 * kSmallWarps);
    }
    mbar_init(ready, 2 * kSmallWarps);
    mbar_init(dready, 2 * kSmallWarps);
    mbar_init(xready, ctas * kSmallWarps);
    mbar_init(drain, 1);
    *abort_flag = 0;
    mbar_fence_init();
    tma_prefetch(&maps.x[0]);
    tma_prefetch(&maps.lo[0]);
  }
  if (warp == 1) {
    tmem_alloc_cg<2>(tmem_slot, 512);
    tmem_relinquish_cg<2>();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  cluster_sync();
  after_previous();

  if (warp == 0) {
    // ------------------------------------------------------ TMA producer
    uint32_t it = 0, steps_done = 0;
    bool ok = true;
    // one box of each CTA into the next slot
    auto load = [&](const CUtensorMap* tm, int y, int z, int mat) {
      const uint32_t slot = it % kSlots, par = (it / kSlots) & 1;
      if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&empty[slot], par ^ 1, abort_flag, sp.err))) return false;
      if (lane == 0) {
        if (rank == 0) mbar_arrive_expect_tx(&full[slot], 2 * kSlotBytes);
        tma_load_4d_pair(ring + slot * kSlotBytes, tm, cluster_addr(&full[slot], lead), 0, y, z, mat);
      }
      __syncwarp();
      ++it;
      return true;
    };
    for (int mat = cid; ok && mat < sp.mats; mat += ncl) {
      for (int s = 0; ok && s < sp.steps; ++s, ++steps_done) {
        const int cur = s & 1;
        if (steps_done > 0) {
          if (!__all_sync(0xFFFFFFFFu, mbar_wait_acquire(xready, (steps_done - 1) & 1, abort_flag, sp.err))) {
            ok = false;
            break;
          }
          fence_proxy_async_global();
        }
        for (int ks = 0; ok && ks < sp.kst_gram; ++ks)
          ok = sp.tall ? load(&maps.x[cur], ks * 128, 2 * rank, mat) : load(&maps.x[cur], 128 * rank, ks * 2, mat);
        for (int tile = pair; ok && tile < sp.tiles; tile += sp.pairs)
          for (int ks = 0; ok && ks < 2 * sp.kst_m; ++ks) {
            const bool low = ks >= sp.kst_m;
            const int k = low ? ks - sp.kst_m : ks;
            const CUtensorMap* tm = low ? &maps.lo[cur] : &maps.x[cur];
            ok = sp.tall ? load(tm, tile * 256 + 128 * rank, k * 2, mat) : load(tm, k * 128, tile * 4 + 2 * rank, mat);
          }
      }
    }
    if (lane == 0 && rank == 0) {
      const uint32_t pend = it < static_cast<uint32_t>(kSlots) ? it : static_cast<uint32_t>(kSlots);
      for (uint32_t j = 0; j < pend; ++j) {
        const uint32_t i2 = it - 1 - j;
        drain_wait(&full[i2 % kSlots], (i2 / kSlots) & 1);
      }
    }
    __syncwarp();
  } else if (warp == 1) {
    if (rank == 0) {
      // ----------------------------------------------------- MMA issuer
      const uint32_t idesc = (1u << 4) | ((256u >> 3) << 17) | ((256u >> 4) << 24);
      const uint32_t gram = idesc | (sp.tall ? kIdescAMnMajor | (1u << 16) : 0u);
      const uint32_t apply = idesc | (sp.tall ? 0u : 1u << 16);
      const uint32_t rg = smem_u32(region);
      uint32_t it = 0, tc = 0, handed = 0;
      bool ok = true;
      auto acquire = [&] {   // an accumulator for the next product
        if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&tempty[tc & 1], ((tc >> 1) & 1) ^ 1, abort_flag, sp.err))) return false;
        tc_fence_after();
        return true;
      };
      auto take = [&] {      // the next slot's boxes
        if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&full[it % kSlots], (it / kSlots) & 1, abort_flag, sp.err))) return false;
        tc_fence_after();
        return true;
      };
      auto stored = [&] {    // A or B is in shared memory
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_acquire(ready, handed & 1, abort_flag, sp.err))) return false;
        ++handed;
        tc_fence_after();
        return true;
      };
      auto done = [&] {
        if (lane == 0) tc_commit_pair_mc(&tfull[tc & 1], both);
        __syncwarp();
        ++tc;
      };
      // 128 contraction elements of a K-major (two chunks from `at`) or MN-major operand
      auto k_major = [](uint32_t at, int j) { return sdesc_k_sw128(at + (j >> 2) * 16384 + (j & 3) * 32); };
      for (int mat = cid; ok && mat < sp.mats; mat += ncl) {
        for (int s = 0; ok && s < sp.steps; ++s) {
          if (!(ok = acquire())) break;
          for (int ks = 0; ks < sp.kst_gram; ++ks, ++it) {
            if (!(ok = take())) break;
            if (lane == 0) {
              const uint32_t sa = smem_u32(ring + (it % kSlots) * kSlotBytes);
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint64_t x = sp.tall ? sdesc_mn_f16(sa + j * 2048) : k_major(sa, j);
                mma_bf16_pair(tmem + (tc & 1) * 256, x, x, gram, (ks | j) ? 1u : 0u);
              }
              tc_commit_pair_mc(&empty[it % kSlots], both);
            }
            __syncwarp();
          }
          if (!ok) break;
          done();
          if (!(ok = stored()) || !(ok = acquire())) break;
          if (lane == 0) {
            for (int ks = 0; ks < sp.kst_m; ++ks) {
#pragma unroll
              for (int j = 0; j < 8; ++j) {
                const uint64_t a = k_major(rg + ks * 32768, j);
                mma_bf16_pair(tmem + (tc & 1) * 256, a, a, idesc, (ks | j) ? 1u : 0u);
              }
            }
          }
          __syncwarp();
          done();
          if (!(ok = stored())) break;
          for (int tile = pair; ok && tile < sp.tiles; tile += sp.pairs) {
            if (!(ok = acquire())) break;
            for (int ks = 0; ks < 2 * sp.kst_m; ++ks, ++it) {
              if (!(ok = take())) break;
              if (lane == 0) {
                const uint32_t sa = smem_u32(ring + (it % kSlots) * kSlotBytes);
                const uint32_t rk = rg + (ks >= sp.kst_m ? ks - sp.kst_m : ks) * 32768;
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  const uint64_t b = k_major(rk, j);
                  const uint64_t x = sp.tall ? k_major(sa, j) : sdesc_mn_f16(sa + j * 2048);
                  mma_bf16_pair(tmem + (tc & 1) * 256, sp.tall ? x : b, sp.tall ? b : x, apply, (ks | j) ? 1u : 0u);
                }
                tc_commit_pair_mc(&empty[it % kSlots], both);
              }
              __syncwarp();
            }
            if (ok) done();
          }
        }
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
    const int lr = q * 32 + lane, r = 128 * rank + lr;   // this lane's row of A and B
    float* ws = turn + (warp - 2) * 1024;
    const uint32_t tempty0 = cluster_addr(tempty, lead);
    const int used = sp.kst_m * 128;                     // columns of A and B that the products read
    uint8_t* mine = region + lr * 128;
    uint32_t tc = 0, steps_done = 0;
    bool ok = true;
    NsParams p{};
    p.rows = sp.rows;
    p.cols = static_cast<int>(sp.pitch);
    p.pitch = sp.pitch;
    p.mat = sp.mat;
    p.diag_n = sp.m;
    p.diag_cols = sp.tall;
    p.o16 = sp.o16;
    p.weight = sp.weight;
    p.w16 = sp.w16;
    p.weight_f32 = sp.weight_f32;
    p.ucols = sp.cols;
    p.decay = sp.decay;
    p.rate = sp.rate;
    p.err = sp.err;
    auto release = [&](uint32_t acc) {   // the accumulator's columns have been read
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive_cluster(tempty0 + 8 * acc);
    };
    auto hand_over = [&] {               // this warp's part of A or B, to the tensor core of its SM
      fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) mbar_arrive_release(ready, lead);
    };
    for (int mat = cid; ok && mat < sp.mats; mat += ncl) {
      for (int s = 0; ok && s < sp.steps; ++s, ++steps_done) {
        const float cb = sp.coef[s][1], cs = sp.coef[s][2] * (1.0f / kSb);
        for (int product = 0; product < 2; ++product, ++tc) {   // A = X X^T, then B = b A + c A A
          const uint32_t acc = tc & 1;
          if (!__all_sync(0xFFFFFFFFu, mbar_wait<true>(&tfull[acc], (tc >> 1) & 1, abort_flag, sp.err))) {
            ok = false;
            break;
          }
          tc_fence_after();
          const uint32_t tbase = tmem + acc * 256 + (static_cast<uint32_t>(q * 32) << 16) + 32 * h;
#pragma unroll 1
          for (int ci = 0; ci < 2; ++ci) {
            const int c0 = 128 * ci + 32 * h;
            if (c0 >= used) continue;
            uint32_t v[32];
            tmem_ld32(tbase + 128 * ci, v);
            tmem_ld_wait();
            uint8_t* chunk = mine + (c0 >> 6) * 16384;
            float dv = 0.0f;
#pragma unroll
            for (int g = 0; g < 4; ++g) {
              uint4* at = reinterpret_cast<uint4*>(chunk + (((((c0 & 63) >> 3) + g) ^ (lr & 7)) << 4));
              float x[8];
#pragma unroll
              for (int j = 0; j < 8; ++j) x[j] = __uint_as_float(v[8 * g + j]);
              if (product == 0) {
#pragma unroll
                for (int j = 0; j < 8; ++j) x[j] *= kSb / (kSx * kSx);
              } else {
                float a[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
                add_half8(*at, a);
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                  x[j] = fmaf(cs, x[j], cb * a[j]);
                  const bool on = c0 + 8 * g + j == r;   // the diagonal goes its own way
                  dv = on ? x[j] : dv;
                  x[j] = on ? 0.0f : x[j];
                }
              }
              *at = make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
            }
            if (product == 1 && c0 == r - lane) {   // in FP32 and in both CTAs
              st_cluster_f32(diag + r, lead, dv * (1.0f / kSb));
              st_cluster_f32(diag + r, lead + 1, dv * (1.0f / kSb));
            }
          }
          release(acc);
          hand_over();
        }
        if (!ok) break;
        if (lane < 2) mbar_arrive_release(dready, lead + lane);
        __syncwarp();
        if (!__all_sync(0xFFFFFFFFu, mbar_wait_acquire(dready, steps_done & 1, abort_flag, sp.err))) {
          ok = false;
          break;
        }
        const int cur = s & 1;
        p.a = sp.coef[s][0];
        p.in_hi = sp.hi[cur];
        p.in_lo = sp.lo[cur];
        p.out_hi = sp.hi[cur ^ 1];
        p.out_lo = sp.lo[cur ^ 1];
        if (s + 1 < sp.steps)
          ok = small_apply<kApply>(sp, p, mat, rank, pair, q, h, lane, ws, tfull, tempty0, tmem, tc, diag, abort_flag);
        else if (sp.o16)
          ok = small_apply<kFinal>(sp, p, mat, rank, pair, q, h, lane, ws, tfull, tempty0, tmem, tc, diag, abort_flag);
        else
          ok = small_apply<kUpdate>(sp, p, mat, rank, pair, q, h, lane, ws, tfull, tempty0, tmem, tc, diag, abort_flag);
        if (!ok) break;
        // this warp's part of the new X, for both CTAs' loads, and its last look at the diagonal
        fence_proxy_async_global();
        __syncwarp();
        if (lane < ctas) mbar_arrive_release(xready, lane);
      }
    }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  cluster_sync();
  if (warp == 1) tmem_dealloc_cg<2>(tmem, 512);
}

}  // namespace

namespace {

const void* small_kernel() { return reinterpret_cast<const void*>(muon_small_kernel); }

// Clusters of 2, 4 and 8 CTAs that the current device runs at a time.
const int* small_clusters() {
  static PerDeviceOnce once;
  static int most[kMaxDevices][3];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return nullptr;
  const cudaError_t e = once.once([&] {
    cudaError_t q = cudaFuncSetAttribute(small_kernel(), cudaFuncAttributeMaxDynamicSharedMemorySize, kSmallSmem);
    for (int i = 0; i < 3 && q == cudaSuccess; ++i) {
      cudaLaunchAttribute at[1];
      at[0].id = cudaLaunchAttributeClusterDimension;
      at[0].val.clusterDim.x = 2 << i;
      at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
      cudaLaunchConfig_t cfg{};
      cfg.gridDim = dim3(2 << i);
      cfg.blockDim = dim3(kSmallThreads);
      cfg.dynamicSmemBytes = kSmallSmem;
      cfg.attrs = at;
      cfg.numAttrs = 1;
      q = cudaOccupancyMaxActiveClusters(&most[dev][i], small_kernel(), &cfg);
    }
    return q;
  });
  return e == cudaSuccess ? most[dev] : nullptr;
}

}  // namespace

// As many pairs as there are tiles, if the device runs clusters of that size
// for all matrices at a time (a second round of clusters costs as much as the
// first).  One tile a pair is always faster than the tiled kernels; with more
// tiles a pair it is the share of busy SMs that decides: from 0.4 of them where
// up to four tiles a pair go through in one round, else from 0.5, or 0.6 where
// m leaves half of the epilogue warps without rows.  Here and tiled: 24 x 256 x
// 2048 (two pairs, 0.63) 231 and 295 us, 16 x 256 x 2048 (0.42) 218 and 235,
// 4 x 256 x 4096 (0.21) 252 and 218, 90 x 256 x 1024 (two rounds, 0.59) 432 and
// 518, 40 x 64 x 4096 (0.53, sixteen tiles a pair) 525 and 462.
int muon_small_pairs(int mats, int m, int k) {
  const int* most = small_clusters();
  if (!most) return 0;
  const int tiles = (k + 255) / 256;
  int i = tiles > 2 ? 2 : tiles > 1 ? 1 : 0;
  for (; i > 0 && mats > most[i];) --i;
  if (most[i] < 1) return 0;
  const int pairs = 1 << i, per = (tiles + pairs - 1) / pairs, rounds = (mats + most[i] - 1) / most[i];
  if (rounds == 1 && per == 1) return pairs;
  const float busy = static_cast<float>(mats) * pairs / (static_cast<float>(rounds) * most[0]);
  return busy >= (rounds == 1 && per <= 4 ? 0.4f : m > 128 ? 0.5f : 0.6f) ? pairs : 0;
}

cudaError_t launch_muon_small(const SmallMaps& maps, const SmallParams& p, cudaStream_t stream) {
  const int* most = small_clusters();
  if (!most) return cudaErrorUnknown;
  void* args[2] = {const_cast<SmallMaps*>(&maps), const_cast<SmallParams*>(&p)};
  const int ctas = 2 * p.pairs, most_now = most[p.pairs == 4 ? 2 : p.pairs - 1];
  return launch_dependent(small_kernel(), dim3(ctas * std::min(most_now, p.mats)), kSmallThreads, kSmallSmem, stream, args, ctas);
}

}  // namespace moe
