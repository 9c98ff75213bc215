// Newton-Schulz products on CTA pairs: what the tiled kernel (muon.cu) and the
// small one (muon_small.cu) share -- stored formats, TMA and descriptors of
// the operands, and the epilogue of a 32 x 32 chunk.  The numbers' design is
// described in muon.cu.
#pragma once

#include <cuda_fp16.h>

#include "kernels.cuh"
#include "moe_gb300.h"

namespace moe {

namespace {

constexpr float kSx = 4096.0f;   // stored X = X * kSx
constexpr float kSb = 512.0f;    // stored A, B = A, B * kSb
constexpr int kThreads = 320;
constexpr int kEpiWarps = 8;
constexpr int kMaxSteps = MOE_MUON_MAX_STEPS;

enum NsKind { kGram, kPoly, kApply, kFinal, kUpdate };   // the last apply: BF16 result, or weight update

struct NsParams {
  int tiles;            // per matrix
  int total;            // tiles of all matrices
  int col_tiles;        // BN-column tiles of the output
  int kstages;          // stages of 128 contraction elements
  int split;            // apply: a second round over them reads X's lo half
  int a_mn, b_mn;       // operand read MN-major
  int rows, cols;       // valid rows, columns written (a multiple of 64)
  int valid_cols;
  long long pitch;      // elements per stored row (multiple of 64)
  long long mat;        // elements per stored matrix
  const __half* in_hi;  // poly: A; apply: X hi
  __half* out_hi;       // gram: A; poly: B; apply: X hi (next)
  const __half* in_lo;  // apply: X lo
  __half* out_lo;       // and where the new one goes (in place unless split)
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
  uint32_t* err;              // a wait that ran out of time; of the products before the last, the run's own word
  const uint32_t* lost;       // last product: that word, nonzero if one of them left its output unfinished
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
  int mat, row0, col0;   // this CTA's 128 output rows, the pair's columns
  int n;                 // columns of the product: BN, or 128 where a last tile needs no more
};

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

// A chunk of FP32 in a warp's 4 KB: 32 rows x 32 columns, or (X) 16 rows x 64
// columns, whose rows are whole 128-byte lines of X's halves: an L1 access
// takes a cycle a line, which halves the loads' and stores' share (3 x 1000 x
// 1531 217 to 210 us, 4 x 1408 x 2048 434 to 418 us).  float4
// slots are spread over the banks: slot j of row r at j ^ (r % 8), or the even
// slots at (j / 2) ^ (r % 8), the odd ones 8 further.
__device__ __forceinline__ int chunk_at(int r, int c) { return r * 32 + ((((c >> 2) ^ (r & 7)) << 2) | (c & 3)); }
__device__ __forceinline__ float4& chunk_quad(float* ws, int r, int quad) {
  return *reinterpret_cast<float4*>(ws + r * 32 + ((quad ^ (r & 7)) << 2));
}
__device__ __forceinline__ int wide_slot(int r, int quad) { return (((quad >> 1) ^ (r & 7)) | ((quad & 1) << 3)) << 2; }
__device__ __forceinline__ float4& wide_quad(float* ws, int r, int quad) {
  return *reinterpret_cast<float4*>(ws + r * 64 + wide_slot(r, quad));
}

// A chunk in its tile.
struct NsChunk {
  int row, col, tcol;   // output row and column, column in the tile
  int half;             // of the quadrant's 32 rows (X)
};

// The chunk's accumulators (tmem: lane quadrant and column of the chunk) to ws.
template <int KIND>
__device__ __forceinline__ void chunk_in(uint32_t tmem, int half, int lane, float* ws) {
#pragma unroll 1
  for (int part = 0; part < (KIND >= kApply ? 2 : 1); ++part) {
    uint32_t v[32];
    tmem_ld32(tmem + 32 * part, v);
    tmem_ld_wait();
    if (KIND < kApply || (lane >> 4) == half) {
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float4 x = make_float4(__uint_as_float(v[4 * j]), __uint_as_float(v[4 * j + 1]),
                                     __uint_as_float(v[4 * j + 2]), __uint_as_float(v[4 * j + 3]));
        if (KIND >= kApply) wide_quad(ws, lane & 15, 8 * part + j) = x;
        else chunk_quad(ws, lane, j) = x;
      }
    }
    __syncwarp();
  }
}

__device__ __forceinline__ void store_half8(__half* p, const float (&x)[8]) {
  *reinterpret_cast<uint4*>(p) =
      make_uint4(pack_half2(x[0], x[1]), pack_half2(x[2], x[3]), pack_half2(x[4], x[5]), pack_half2(x[6], x[7]));
}
__device__ __forceinline__ void add_half8(const uint4& u, float (&x)[8]) {
  const uint32_t h[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    x[2 * j] += half_lo(h[j]);
    x[2 * j + 1] += half_hi(h[j]);
  }
}

__device__ __forceinline__ uint4 pack_bf16x8(const float (&x)[8], float s) {
  return make_uint4(pack_bf16x2(x[0] * s, x[1] * s), pack_bf16x2(x[2] * s, x[3] * s), pack_bf16x2(x[4] * s, x[5] * s),
                    pack_bf16x2(x[6] * s, x[7] * s));
}

// 8 values of the caller's weight from element u (x: the new X, stored
// scale; w4: the weight there).  16-byte accesses.
__device__ __forceinline__ void put_weight8(const NsParams& p, long long u, const float (&x)[8], const uint4 (&w4)[2]) {
  const float rate = -p.rate * (1.0f / kSx);
  float w[8];
  if (p.weight_f32) {
    const uint32_t q[8] = {w4[0].x, w4[0].y, w4[0].z, w4[0].w, w4[1].x, w4[1].y, w4[1].z, w4[1].w};
#pragma unroll
    for (int j = 0; j < 8; ++j) w[j] = fmaf(p.decay, __uint_as_float(q[j]), rate * x[j]);
    float4* o = reinterpret_cast<float4*>(static_cast<float*>(p.weight) + u);
    o[0] = make_float4(w[0], w[1], w[2], w[3]);
    o[1] = make_float4(w[4], w[5], w[6], w[7]);
    if (p.w16) *reinterpret_cast<uint4*>(p.w16 + u) = pack_bf16x8(w, 1.0f);
  } else {
    const uint32_t q[4] = {w4[0].x, w4[0].y, w4[0].z, w4[0].w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[2 * j] = fmaf(p.decay, bf16_lo(q[j]), rate * x[2 * j]);
      w[2 * j + 1] = fmaf(p.decay, bf16_hi(q[j]), rate * x[2 * j + 1]);
    }
    *reinterpret_cast<uint4*>(static_cast<__nv_bfloat16*>(p.weight) + u) = pack_bf16x8(w, 1.0f);
  }
}
// One value, where rows start anywhere; w: the weight there.
__device__ __forceinline__ void put_update1(const NsParams& p, long long u, float x, float w) {
  w = fmaf(p.decay, w, -p.rate * (1.0f / kSx) * x);
  if (p.weight_f32) static_cast<float*>(p.weight)[u] = w;
  else static_cast<__nv_bfloat16*>(p.weight)[u] = __float2bfloat16_rn(w);
  if (p.w16) p.w16[u] = __float2bfloat16_rn(w);
}

// What a chunk needs besides the accumulator: 8 columns of four rows a lane.
// All of a chunk's loads are sent together: refilling the registers row by row
// as they are used, two chunks ahead, was slower (an apply product of 8 x 7168
// x 2048 404 instead of 310 us), since a warp waits on few counters of loads
// in flight and then waits for the youngest of those that share one.
// LATE: the weight follows when the chunk is worked on.
template <int KIND, bool LATE = false>
struct ChunkIn {
  uint4 hi[4], lo[4];
  uint4 w[KIND == kUpdate && !LATE ? 4 : 1][2];   // the weight (rows that vectors divide)
};

// 8 columns of the caller's weight.
__device__ __forceinline__ void load_weight8(const NsParams& p, int mat, int r, int c, uint4 (&w)[2]) {
  if (p.ucols % 8 == 0 && r < p.rows && c < p.ucols) {
    const long long u = (static_cast<long long>(mat) * p.rows + r) * p.ucols + c;
    if (p.weight_f32) {
      w[0] = reinterpret_cast<const uint4*>(static_cast<const float*>(p.weight) + u)[0];
      w[1] = reinterpret_cast<const uint4*>(static_cast<const float*>(p.weight) + u)[1];
    } else {
      w[0] = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p.weight) + u);
    }
  }
}

template <int KIND, bool LATE>
__device__ __forceinline__ void load_chunk_in(const NsParams& p, int mat, int r0, int c0, int lane, ChunkIn<KIND, LATE>& in) {
  if constexpr (KIND == kGram) return;
  constexpr int kLanes = KIND >= kApply ? 8 : 4;   // of a row
  const int c = c0 + (lane % kLanes) * 8;
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int r = r0 + it * (32 / kLanes) + lane / kLanes;
    in.hi[it] = in.lo[it] = make_uint4(0, 0, 0, 0);
    if (r < p.rows && c < p.cols) {
      const long long at = mat * p.mat + r * p.pitch + c;
      in.hi[it] = *reinterpret_cast<const uint4*>(p.in_hi + at);
      if constexpr (KIND >= kApply) in.lo[it] = *reinterpret_cast<const uint4*>(p.in_lo + at);
    }
    if constexpr (KIND == kUpdate && !LATE) load_weight8(p, mat, r, c, in.w[it]);
  }
}

// The chunk at rows r0, columns c0, whose accumulator values are in ws.  A
// lane takes 8 columns of a row at a time.  d: the matrix's diagonal of B
// (apply).
template <int KIND, bool LATE>
__device__ __forceinline__ void ns_chunk(const NsParams& p, const NsTile& t, int r0, int c0, int lane, float* ws,
                                         const ChunkIn<KIND, LATE>& in, const float* d) {
  constexpr int kLanes = KIND >= kApply ? 8 : 4;   // of a row
  const int quad = (lane % kLanes) * 2, c = c0 + (lane % kLanes) * 8;
  const bool mirror = (KIND == kGram || KIND == kPoly) && (c0 >> 7) > (r0 >> 7);
#pragma unroll
  for (int it = 0; it < 4; ++it) {
    const int rr = it * (32 / kLanes) + lane / kLanes, r = r0 + rr;
    const float4 a = KIND >= kApply ? wide_quad(ws, rr, quad) : chunk_quad(ws, rr, quad);
    const float4 b = KIND >= kApply ? wide_quad(ws, rr, quad + 1) : chunk_quad(ws, rr, quad + 1);
    float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    const bool inside = r < p.rows && c < p.cols;
    const long long at = t.mat * p.mat + r * p.pitch + c;
    if constexpr (KIND == kGram) {
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] *= kSb / (kSx * kSx);
      if (inside) store_half8(p.out_hi + at, x);
    } else if constexpr (KIND == kPoly) {
      const float cs = p.c * (1.0f / kSb);
      float g[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      add_half8(in.hi[it], g);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        x[j] = fmaf(cs, x[j], p.b * g[j]);
        if (c + j == r) {
          if (r < p.rows) p.diag[static_cast<long long>(t.mat) * p.diag_n + r] = x[j] * (1.0f / kSb);
          x[j] = 0.0f;
        }
      }
      if (inside) store_half8(p.out_hi + at, x);
      if (mirror) {
        chunk_quad(ws, rr, quad) = make_float4(x[0], x[1], x[2], x[3]);
        chunk_quad(ws, rr, quad + 1) = make_float4(x[4], x[5], x[6], x[7]);
      }
    } else {
      float g[8] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      add_half8(in.hi[it], g);
      add_half8(in.lo[it], g);
      if (p.diag_cols) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float dj = c + j < p.diag_n ? d[c + j] : 0.0f;
          x[j] = fmaf(p.a + dj, g[j], x[j] * (1.0f / kSb));
        }
      } else {
        const float f = p.a + (r < p.rows ? d[r] : 0.0f);
#pragma unroll
        for (int j = 0; j < 8; ++j) x[j] = fmaf(f, g[j], x[j] * (1.0f / kSb));
      }
      if constexpr (KIND == kApply) {
        if (inside) store_hi_lo(p.out_hi + at, p.out_lo + at, x);
      } else if (p.ucols % 8 == 0) {
        if (inside && c < p.ucols) {
          const long long u = (static_cast<long long>(t.mat) * p.rows + r) * p.ucols + c;
          if constexpr (KIND == kFinal) *reinterpret_cast<uint4*>(p.o16 + u) = pack_bf16x8(x, 1.0f / kSx);
          else if constexpr (!LATE) {
            put_weight8(p, u, x, in.w[it]);
          } else {
            uint4 w[2];
            load_weight8(p, t.mat, r, c, w);
            put_weight8(p, u, x, w);
          }
        }
      } else {
        wide_quad(ws, rr, quad) = make_float4(x[0], x[1], x[2], x[3]);
        wide_quad(ws, rr, quad + 1) = make_float4(x[4], x[5], x[6], x[7]);
      }
    }
  }
  if (KIND >= kFinal && p.ucols % 8 != 0) {
    // rows that no vector divides: a lane two columns of four rows at a time,
    // whose weights are all asked for before the first is written (one by one
    // the last product of 40 x 63 x 7169 took 1027 us instead of 552)
    __syncwarp();
#pragma unroll 1
    for (int rb = 0; rb < 16; rb += 4) {
      float w[8];
      auto weights = [&](const auto* from) {
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          const int r = r0 + rb + (k >> 1), cc = c0 + lane + 32 * (k & 1);
          w[k] = 0.0f;
          if (r < p.rows && cc < p.ucols)
            w[k] = static_cast<float>(from[(static_cast<long long>(t.mat) * p.rows + r) * p.ucols + cc]);
        }
      };
      if constexpr (KIND == kUpdate) {
        if (p.weight_f32) weights(static_cast<const float*>(p.weight));
        else weights(static_cast<const __nv_bfloat16*>(p.weight));
      }
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const int rr = rb + (k >> 1), r = r0 + rr, c1 = lane + 32 * (k & 1), cc = c0 + c1;
        if (r < p.rows && cc < p.ucols) {
          const long long u = (static_cast<long long>(t.mat) * p.rows + r) * p.ucols + cc;
          const float x1 = ws[rr * 64 + wide_slot(rr, c1 >> 2) + (c1 & 3)];
          if constexpr (KIND == kUpdate) put_update1(p, u, x1, w[k]);
          else p.o16[u] = __float2bfloat16_rn(x1 * (1.0f / kSx));
        }
      }
    }
  }
  if (mirror) {   // rows c0 .. c0 + 31 of the image, columns r0 .. r0 + 31
    __syncwarp();
    const int col = r0 + (lane & 3) * 8;
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int rr = it * 8 + (lane >> 2), r = c0 + rr;
      float x[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) x[j] = ws[chunk_at((lane & 3) * 8 + j, rr)] * (KIND == kGram ? kSb / (kSx * kSx) : 1.0f);
      if (r < p.rows && col < p.cols) store_half8(p.out_hi + t.mat * p.mat + r * p.pitch + col, x);
    }
  }
  __syncwarp();   // the chunk has been read
}

__device__ __forceinline__ void drain_wait(uint64_t* bar, uint32_t parity) {
  const long long t0 = clock64();
  while (!mbar_try_wait(bar, parity)) {
    if (clock64() - t0 > kWaitTimeoutCycles / 8) return;
  }
}

}  // namespace

// The small kernel: all steps of each matrix on a few CTA pairs (m <= 256).
struct SmallMaps {
  CUtensorMap x[2], lo[2];   // X's halves (both buffers): 128 rows of two 64-column chunks
};
struct SmallParams {
  int mats, steps;
  int pairs;                 // per matrix (1, 2 or 4), a cluster
  int tall;
  int kst_gram, kst_m;       // stages of 128 contraction elements: over k, over m
  int tiles;                 // 256-row (tall) or 256-column tiles of X
  int m, rows, cols;
  long long pitch, mat;      // stored X
  __half* hi[2];
  __half* lo[2];
  float coef[MOE_MUON_MAX_STEPS][3];
  __nv_bfloat16* o16;
  void* weight;
  __nv_bfloat16* w16;
  int weight_f32;
  float decay, rate;
  uint32_t* err;
};
// Pairs per matrix for `mats` matrices of sizes m <= k, or 0: the tiled
// kernels are the faster ones.
int muon_small_pairs(int mats, int m, int k);
cudaError_t launch_muon_small(const SmallMaps& maps, const SmallParams& p, cudaStream_t stream);

}  // namespace moe
