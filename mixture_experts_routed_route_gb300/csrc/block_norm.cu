// Norms around a block with its gate and the scaled residual, in one pass,
// and their backward (moe_block_norm_forward / _backward).
//
//   n = o r_o,  r_o = 1/sqrt(mean o^2 + eps)          (norm after the block)
//   y = alpha x + beta g n w_o                        (gate, residual)
//   h = y r_y w_h,  r_y = 1/sqrt(mean y^2 + eps)      (norm before the next)
//
// with w = weight + weight_offset.  h is formed from the unrounded FP32 y,
// and the backward rebuilds that same y from x and o (as many bytes as
// reading the rounded y back), so forward and backward agree to FP32.
// Gradients, with z = y r_y, a = dh w_h and sums over the row's D columns:
//   s  = dy + r_y (a - z mean(a z))                   (gradient of y)
//   dx = alpha s,   dg = beta s n w_o,   b = beta g s w_o
//   do = r_o (b - n mean(b n)),  dw_o = sum_t beta g s n,  dw_h = sum_t dh z
//
// Work layout: persistent CTAs, one per SM.  A group of W warps owns a row
// (W = ceil(D / 1024) with 32 columns a thread in four pieces of 8, or twice
// as many with half of that); as many groups share a CTA as its registers and
// shared memory hold, and take rows in turns over the CTAs.  Rows come in
// through shared memory, cp.async, and are read from there once per pass
// over them (the row's sums separate the passes), so registers hold only
// what a later pass needs: the FP32 y in the forward; in the backward the
// running column sums and one value a column.  Several small groups rather
// than one of the whole CTA: while one waits for its row or at its named
// barrier the others issue, and 32 columns a thread carry the fixed cost of
// a row (two sums over the warps, the copies, the bookkeeping).
//   V = 8: rows whose length and strides are multiples of 8 elements; a
//          thread copies just the 16-byte pieces it will read itself, so the
//          copies need no barrier.
//   V = 1: any other row; the group copies the aligned 16-byte pieces that
//          cover it and reads its elements at the row's own offset, between
//          two more barriers.
//
// What it measures (BF16, channel gate or none, of 6.77 TB/s measured):
// forward 2048 x 7168 24.4 us (4.8 TB/s), 8192 x 7168 82 us (5.7), FP32
// residual with a gate row a sequence 16384 x 2048 70 us (5.8); backward 2048 x 7168
// 46 us (3.8), 8192 x 7168 137 us (5.1), 1531 x 1411 in FP32 with a token gate 23 us (1.7).
// Gates that change by the row keep more of it alive, and their backward
// spills (208 to 224 bytes of stores with vector rows, 472 without, and 52 to
// 60, 268 for a gate of every element): 2048 x 7168 with eight gate rows 70 us
// and with a gate of every element 83, FP32 16384 x 2048 with eight gate rows
// 143 us where a channel gate takes 112, 1532 x 1411 with four 60 us.  Widths
// that no vector divides, forward: 1531 x 1411 in FP32 12.4 us (2.1 TB/s),
// BF16 16384 x 1411 78 us (2.4).
// Long inputs are bound by the stream; short ones by the fixed part (launch,
// factors, column sums: 7 us forward, 15 us backward with its second kernel)
// and the backward by latency inside a row: its three passes and two sums are
// one chain, 14 warps issue in 43 % of the cycles, and registers (column
// sums) leave no room for a second row beside them.  Tried there without
// gain: factors in registers instead of the table (spills, which go to L2
// beside this much shared memory: 65 us), 28 warps with one piece each (65),
// z formed twice instead of kept (46.5), a dependent launch of the second
// kernel (as fast on the device, 2 us more on the host), 512 threads in it.
#include <algorithm>

#include "kernels.cuh"
#include "moe_gb300.h"

namespace moe {

namespace {

constexpr int kMaxCols = 8192;           // the table and one row of every stream fit beside each other
constexpr int kSharedMem = 216 * 1024;   // the columns' factors and the rows in flight
constexpr int kWarps = 16;            // of a CTA at most: 128 registers a thread

// A tensor whose rows the kernel streams.
struct Stream {
  const uint8_t* base;        // NULL: not there
  long long ld;               // bytes between rows
  const uint8_t* end;         // past the last row's last element
  int esz, row_bytes;
  int off;                    // place in a row's slot
  int piece;                  // bytes between a thread's 8-column pieces (V = 8)
};
enum { kX, kDy, kDh, kG, kO, kStreams };   // kG: a gate of every element; kO: what the backward reads last

// gate_mode inside: a grouped gate whose groups are single rows is a gate of
// every element, which is streamed like x and has no sums over rows.
constexpr int kGateFull = MOE_GATE_TOKEN + 1;

struct NormParams {
  int T, D;
  int warps, groups;          // warps per row, rows in flight per CTA
  int stages, slot;           // rows in flight per group, bytes of one
  int table;                  // bytes of the columns' factors
  int res_f32;                // residual type
  Stream in[kStreams];
  const void* gate;
  const void* w_post;         // NULL: no norm after the block
  const void* w_pre;          // NULL: no norm before the next
  long long ldy, ldh;
  int gate_mode, rows_per_group;
  int params_f32, gate_f32;
  float alpha, beta, eps, offset;
  // forward
  void* y;
  __nv_bfloat16* h;
  float* stats;               // [2][T]: r_o, r_y (backward: read)
  // backward
  void* dx;                   // or NULL
  __nv_bfloat16* do_;
  void* dgate;
  float* partial;             // [2][gridDim.x][D]: sum s n (times g: grouped, token gates, gates of every element), sum dh z
  float* gate_partial;        // [slabs][D] (grouped gates cut into several slabs a group)
  int slabs_per_group, slabs;
};

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// Two FP32 operations an instruction (packed f32x2): the passes below are
// bound by instruction issue as soon as the rows stream at full rate.
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
__device__ __forceinline__ unsigned long long mul2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ unsigned long long add2(unsigned long long a, unsigned long long b) {
  unsigned long long r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(unsigned long long v) {
  float a, b;
  split(v, a, b);
  return a + b;
}

using Pair = unsigned long long;
__device__ __forceinline__ Pair both(float x) { return pair_of(x, x); }

// V of the kernels: 8 (vector rows), 1 (any row), or kFull: vector rows whose
// D is a multiple of 1024, so that no column needs a test.
constexpr int kFull = 16;

// Pieces of 8 columns a thread holds: two in the backward, whose column sums
// stay in registers too (four: 70 us instead of 51 at 2048 x 7168, with
// half the warps and spills), and where every column has its own address and
// test (V = 1).
template <int V, bool BWD>
constexpr int kPiecesOf = (V == 1 || BWD) ? 2 : 4;

// A thread's 32 columns of its group's row in pieces i of 8: neighbours
// (vector rows) or nt apart (V = 1).
template <int V>
struct Columns {
  int t, nt, D;
  __device__ __forceinline__ int col(int i, int j) const { return V >= 8 ? (t + i * nt) * 8 + j : t + (8 * i + j) * nt; }
  __device__ __forceinline__ bool any(int i) const { return V == kFull || col(i, 0) < D; }

  // piece i of a row, as pairs; zeros past D
  __device__ __forceinline__ void load(const __nv_bfloat16* row, int i, Pair (&q)[4]) const {
    if constexpr (V >= 8) {
      uint4 u = make_uint4(0, 0, 0, 0);
      if (any(i)) u = *reinterpret_cast<const uint4*>(row + col(i, 0));
      q[0] = pair_of(bf16_lo(u.x), bf16_hi(u.x));
      q[1] = pair_of(bf16_lo(u.y), bf16_hi(u.y));
      q[2] = pair_of(bf16_lo(u.z), bf16_hi(u.z));
      q[3] = pair_of(bf16_lo(u.w), bf16_hi(u.w));
    } else {
      scalars(row, i, q);
    }
  }
  __device__ __forceinline__ void load(const float* row, int i, Pair (&q)[4]) const {
    if constexpr (V >= 8) {
      float4 a = make_float4(0.0f, 0.0f, 0.0f, 0.0f), b = a;
      if (any(i)) {
        a = *reinterpret_cast<const float4*>(row + col(i, 0));
        b = *reinterpret_cast<const float4*>(row + col(i, 4));
      }
      q[0] = pair_of(a.x, a.y);
      q[1] = pair_of(a.z, a.w);
      q[2] = pair_of(b.x, b.y);
      q[3] = pair_of(b.z, b.w);
    } else {
      scalars(row, i, q);
    }
  }
  template <typename X>
  __device__ __forceinline__ void scalars(const X* row, int i, Pair (&q)[4]) const {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = col(i, j) < D ? to_f(row[col(i, j)]) : 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) q[j] = pair_of(v[2 * j], v[2 * j + 1]);
  }
  __device__ __forceinline__ void load(const void* row, int f32, int i, Pair (&q)[4]) const {
    if (f32) load(static_cast<const float*>(row), i, q);
    else load(static_cast<const __nv_bfloat16*>(row), i, q);
  }

  template <typename X>
  __device__ __forceinline__ void store(X* row, int i, const Pair (&q)[4]) const {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) split(q[j], v[2 * j], v[2 * j + 1]);
    if constexpr (V >= 8) {
      if (!any(i)) return;
      if constexpr (sizeof(X) == 2) {
        *reinterpret_cast<uint4*>(row + col(i, 0)) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                                                pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
      } else {
        *reinterpret_cast<float4*>(row + col(i, 0)) = make_float4(v[0], v[1], v[2], v[3]);
        *reinterpret_cast<float4*>(row + col(i, 4)) = make_float4(v[4], v[5], v[6], v[7]);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (col(i, j) < D) put(row + col(i, j), v[j]);
    }
  }
  __device__ __forceinline__ void store(void* row, int f32, int i, const Pair (&q)[4]) const {
    if (f32) store(static_cast<float*>(row), i, q);
    else store(static_cast<__nv_bfloat16*>(row), i, q);
  }
};

// One value of either type.
__device__ __forceinline__ float param_at(const void* p, int f32, long long i) {
  return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}
__device__ __forceinline__ void param_put(void* p, int f32, long long i, float v) {
  if (f32) static_cast<float*>(p)[i] = v;
  else static_cast<__nv_bfloat16*>(p)[i] = __float2bfloat16_rn(v);
}
__device__ __forceinline__ const void* param_row(const void* p, int f32, long long i) {
  return static_cast<const uint8_t*>(p) + i * (f32 ? 4 : 2);
}
__device__ __forceinline__ void* param_row(void* p, int f32, long long i) {
  return static_cast<uint8_t*>(p) + i * (f32 ? 4 : 2);
}

// 1/sqrt(x): the hardware's approximation and one Newton step.
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return r < INFINITY && r > 0.0f ? r * fmaf(-0.5f * x * r, r, 1.5f) : r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// the first `bytes` of 16, zeros after them
__device__ __forceinline__ void cp_async16(uint32_t dst, const uint8_t* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// 8 values of a weight or gate [D] from column c (16-byte aligned whatever D is).
__device__ __forceinline__ void params8(const void* p, int f32, int c, int D, float (&v)[8]) {
  if (c + 8 <= D) {
    if (f32) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c));
      const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c) + 1);
      v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
    } else {
      const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + c));
      v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
      v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
    }
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = c + j < D ? param_at(p, f32, c + j) : 0.0f;
  }
}

__device__ __forceinline__ float token_gate(const NormParams& p, long long row) {
  return p.gate_mode == MOE_GATE_TOKEN ? param_at(p.gate, p.gate_f32, row) : 1.0f;
}

// A group of warps: its place, its columns' factors and its rows in flight.
template <int V, int P>
struct Group {
  const NormParams& p;
  Columns<V> cols;
  int grp, wig, bar;
  float* red;
  int turn = 0;
  const float* table;     // f [D], w_pre [D]
  uint8_t* slots;
  long long next_row, step;
  int left, fill;         // rows still to send for, and the slot of the next
  int take;               // slot of the row at hand

  __device__ __forceinline__ Group(const NormParams& p_, uint8_t* shared, float (*red_all)[64]) : p(p_) {
    const int warp = threadIdx.x >> 5;
    grp = warp / p.warps;
    wig = warp - grp * p.warps;
    cols.nt = p.warps * 32;
    cols.t = threadIdx.x - grp * cols.nt;
    cols.D = p.D;
    bar = 1 + grp;
    red = red_all[grp];
    for (int i = threadIdx.x; i < 15 * 64; i += blockDim.x) (&red_all[0][0])[i] = 0.0f;
    table = reinterpret_cast<const float*>(shared);
    slots = shared + p.table + static_cast<size_t>(grp) * p.stages * p.slot;
  }

  // Fill the CTA's table with what the weights and a channel gate contribute
  // to each column: f = beta w_post g, the factor of n in y, and w_pre (all
  // threads; ends with a barrier).
  __device__ __forceinline__ void make_table(uint8_t* shared) const {
    float* f = reinterpret_cast<float*>(shared);
    float* h = f + p.table / 8;
    for (int c = threadIdx.x * 8; c < p.D; c += blockDim.x * 8) {
      float a[8], b[8], w[8];
      if (p.w_post) params8(p.w_post, p.params_f32, c, p.D, a);
      if (p.gate_mode == MOE_GATE_CHANNEL) params8(p.gate, p.gate_f32, c, p.D, b);
      if (p.w_pre) params8(p.w_pre, p.params_f32, c, p.D, w);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        float v = p.beta;
        if (p.w_post) v *= a[j] + p.offset;
        if (p.gate_mode == MOE_GATE_CHANNEL) v *= b[j];
        if (c + j < p.D) {
          f[c + j] = v;
          h[c + j] = p.w_pre ? w[j] + p.offset : 0.0f;
        }
      }
    }
    __syncthreads();
  }
  __device__ __forceinline__ void factor(int which, int i, Pair (&q)[4]) const {
    cols.load(table + which * (p.table / 8), i, q);
  }

  __device__ __forceinline__ void sync() const {
    if (p.warps == 1) __syncwarp();
    else named_bar_sync(bar, cols.nt);
  }

  // Sum over the group in a fixed order: an xor tree in each warp, then the
  // warp sums in quads.  `red` is 2 x 32 floats (zero beyond the warps),
  // used in turns, so one barrier a sum is enough.
  __device__ __forceinline__ float sum(Pair v2) {
    float v = sum2(v2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (p.warps == 1) return v;
    float* r = red + turn;
    turn ^= 32;
    if ((threadIdx.x & 31) == 0) r[wig] = v;
    named_bar_sync(bar, cols.nt);
    return warp_sums(r);
  }
  __device__ __forceinline__ float warp_sums(const float* r) const {
    const float4* q = reinterpret_cast<const float4*>(r);
    float t = (q[0].x + q[0].y) + (q[0].z + q[0].w);
    if (p.warps > 4) t += (q[1].x + q[1].y) + (q[1].z + q[1].w);
    if (p.warps > 8) t += ((q[2].x + q[2].y) + (q[2].z + q[2].w)) + ((q[3].x + q[3].y) + (q[3].z + q[3].w));
    return t;
  }

  // Two sums at once.
  __device__ __forceinline__ void sum_two(Pair a2, Pair b2, float& sa, float& sb) {
    float a = sum2(a2), b = sum2(b2);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (p.warps == 1) {
      sa = a;
      sb = b;
      return;
    }
    float* r = red + turn;
    turn ^= 32;
    if ((threadIdx.x & 31) == 0) {
      r[wig] = a;
      r[16 + wig] = b;
    }
    named_bar_sync(bar, cols.nt);
    sa = warp_sums(r);
    sb = warp_sums(r + 16);
  }

  // Copy the next row's streams LO .. HI - 1 into slot `fill`.
  template <int LO, int HI>
  __device__ __forceinline__ void copy() const {
    const uint32_t slot = smem_u32(slots) + fill * p.slot;
#pragma unroll
    for (int k = LO; k < HI; ++k) {
      if (p.in[k].base == nullptr) continue;
      const uint8_t* src = p.in[k].base + next_row * p.in[k].ld;
      uint32_t dst = slot + p.in[k].off;
      if constexpr (V >= 8) {
        // this thread's own columns: 8 elements are 16 or 32 bytes
        const int at = cols.t * 8 * p.in[k].esz;
        src += at;
        dst += at;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (cols.any(i)) {
            cp_async16(dst + i * p.in[k].piece, src + i * p.in[k].piece);
            if (p.in[k].esz == 4) cp_async16(dst + i * p.in[k].piece + 16, src + i * p.in[k].piece + 16);
          }
        }
      } else {
        const uint8_t* a = src - (reinterpret_cast<uintptr_t>(src) & 15);
        const int n = static_cast<int>(src - a + p.in[k].row_bytes + 15) >> 4;
        const long long all = p.in[k].end - a;   // 16 n passes it in the last row only
        for (int j = cols.t; j < n; j += cols.nt) {
          const long long rest = all - 16ll * j;
          cp_async16(dst + 16 * j, a + 16ll * j, rest < 16 ? static_cast<int>(rest) : 16);
        }
      }
    }
  }
  __device__ __forceinline__ void sent() {
    next_row += step;
    --left;
    fill = fill + 1 == p.stages ? 0 : fill + 1;
  }

  // Send for the first rows of first, first + step, ... (n of them).
  __device__ __forceinline__ void start(long long first, long long step_, int n) {
    next_row = first;
    step = step_;
    left = n;
    fill = 0;
    take = -1;
    for (int i = 0; i < p.stages; ++i) {
      if (left > 0) {
        copy<0, kStreams>();
        sent();
      }
      cp_commit();
    }
  }
  // Make the next row ready; its slot.  HELD: the row before it has not been
  // released yet.
  template <bool HELD>
  __device__ __forceinline__ int next() {
    take = take + 1 == p.stages ? 0 : take + 1;
    const int newer = p.stages - 1 - HELD;   // rows that may still be under way
    if (newer <= 0) cp_wait<0>();
    else if (newer == 1) cp_wait<1>();
    else if (newer == 2) cp_wait<2>();
    else cp_wait<3>();
    if (V == 1) sync();
    return take;
  }
  // The oldest row has been read (early: all of it but o, where a thread
  // reads what it copied itself): its place takes the row `stages` further on.
  __device__ __forceinline__ void release_early() {
    if (V >= 8 && left > 0) copy<0, kO>();
  }
  __device__ __forceinline__ void release() {
    if (left > 0) {
      if (V == 1) sync();
      copy<V >= 8 ? kO : 0, kStreams>();
      sent();
    }
    cp_commit();
  }

  template <typename X = void>
  __device__ __forceinline__ const X* stream(int k, long long row, int slot) const {
    const uint8_t* q = slots + slot * p.slot + p.in[k].off;
    if constexpr (V == 1) q += reinterpret_cast<uintptr_t>(p.in[k].base + row * p.in[k].ld) & 15;
    return reinterpret_cast<const X*>(q);
  }
  // The row's own gate (grouped gates and gates of every element).
  __device__ __forceinline__ const void* gate_row(long long row, int slot) const {
    if (p.in[kG].base) return stream(kG, row, slot);
    return param_row(p.gate, p.gate_f32, static_cast<long long>(static_cast<uint32_t>(row) / static_cast<uint32_t>(p.rows_per_group)) * p.D);
  }
};

template <typename R, int V, bool ALL>
__global__ void __launch_bounds__(kWarps * 32, 1) block_norm_fwd_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) float red_all[15][64];
  constexpr int P = kPiecesOf<V, false>;
  Group<V, P> g(p, shared, red_all);
  const int first = g.grp * gridDim.x + blockIdx.x, step = gridDim.x * p.groups;
  const int n = first < p.T ? (p.T - 1 - first) / step + 1 : 0;
  g.start(first, step, n);
  g.make_table(shared);
  const Columns<V> cols = g.cols;
  // ALL: every part is there and no gate changes by the row (the common call)
  const bool has_o = ALL || p.in[kO].base != nullptr, post = ALL || p.w_post != nullptr, pre = ALL || p.w_pre != nullptr;
  const bool row_gate = !ALL && (p.gate_mode == MOE_GATE_GROUP || p.gate_mode == kGateFull);
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const Pair alpha = both(p.alpha);
  long long row = first;
  for (int it = 0; it < n; ++it, row += step) {
    const int slot = g.template next<false>();
    Pair y[P][4], o[P][4];
    float r_o = 1.0f;
    if (has_o) {
      const __nv_bfloat16* os = g.template stream<__nv_bfloat16>(kO, row, slot);
      Pair so = both(0.0f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (V >= 8 && !cols.any(i)) continue;
        Pair f[4];
        cols.load(os, i, o[i]);
        g.factor(0, i, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          so = fma2(o[i][j], o[i][j], so);
          o[i][j] = mul2(o[i][j], f[j]);
        }
      }
      if (row_gate) {
        const void* gr = g.gate_row(row, slot);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (V >= 8 && !cols.any(i)) continue;
          Pair f[4];
          cols.load(gr, p.gate_f32, i, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) o[i][j] = mul2(o[i][j], f[j]);
        }
      }
      if (post) {
        r_o = inv_sqrt(fmaf(g.sum(so), inv_d, p.eps));
        if (p.stats && cols.t == 0) p.stats[row] = r_o;
      }
      r_o *= token_gate(p, row);
    }
    const R* xs = g.template stream<R>(kX, row, slot);
    const Pair r2 = both(r_o);
    Pair sy = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (V >= 8 && !cols.any(i)) continue;
      cols.load(xs, i, y[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        y[i][j] = mul2(alpha, y[i][j]);
        if (has_o) y[i][j] = fma2(o[i][j], r2, y[i][j]);
        sy = fma2(y[i][j], y[i][j], sy);
      }
      if (ALL || p.y) cols.store(static_cast<R*>(p.y) + row * p.ldy, i, y[i]);
    }
    g.release_early();
    g.release();
    if (pre) {
      const float r_y = inv_sqrt(fmaf(g.sum(sy), inv_d, p.eps));
      if (p.stats && cols.t == 0) p.stats[p.T + row] = r_y;
      const Pair ry2 = both(r_y);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (V >= 8 && !cols.any(i)) continue;
        Pair w[4];
        g.factor(1, i, w);
#pragma unroll
        for (int j = 0; j < 4; ++j) w[j] = mul2(mul2(y[i][j], ry2), w[j]);
        cols.store(p.h + row * p.ldh, i, w);
      }
    }
  }
  cp_wait<0>();
}

// A group's rows: every gridDim * groups-th one, or (grouped gates) the
// slabs it owns, each within one gate row.  With f = beta g w_o, y = alpha x
// + f n and b = f s, so one factor a column serves both directions; and the
// parameter sums need only S = sum_t s n a column (dw_o = beta g S, dgate =
// beta w_o S where g does not change with t) and sum_t dh z.  They stay in
// registers (GATE is MOE_GATE_NONE for every gate that needs no more than
// that) and are added over the CTA's groups, in group order, at the end; a
// grouped gate's S is turned into its dgate, and into dw_o, slab by slab.
// Passes over a row in shared memory: x, o, dh for sum a z; then dh, dy, o
// for s, dx and b (z, kept, gives its place to b); then o for do.
template <typename R, int V, int GATE, bool ALL>
__global__ void __launch_bounds__(kWarps * 32, 1) block_norm_bwd_kernel(const __grid_constant__ NormParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) float red_all[15][64];
  constexpr int P = kPiecesOf<V, true>;
  Group<V, P> g(p, shared, red_all);
  const int worker = g.grp * gridDim.x + blockIdx.x, workers = gridDim.x * p.groups;
  if constexpr (GATE != MOE_GATE_GROUP) {
    g.start(worker, workers, worker < p.T ? (p.T - 1 - worker) / workers + 1 : 0);
  }
  g.make_table(shared);
  const Columns<V> cols = g.cols;
  // ALL: every part is there (the common call), which these tests then cost nothing
  const bool has_o = ALL || p.in[kO].base != nullptr, has_dy = ALL || p.in[kDy].base != nullptr;
  const bool post = ALL || p.w_post != nullptr, pre = ALL || p.w_pre != nullptr, has_dx = ALL || p.dx != nullptr;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  Pair S[P][4], aw_h[P][4];   // running column sums
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) S[i][j] = aw_h[i][j] = both(0.0f);

  // a row's statistics and token gate, loaded a row before they are needed
  struct RowStats {
    float r_o, r_y, tg;
  };
  auto stats_of = [&](long long row) {
    RowStats q;
    q.r_o = (has_o && post) ? p.stats[row] : 1.0f;
    q.r_y = pre ? p.stats[p.T + row] : 0.0f;
    q.tg = has_o ? token_gate(p, row) : 1.0f;
    return q;
  };
  // the row in ring slot `slot`: z = y r_y, sum_t dh z, and this thread's part of sum a z
  auto first_pass = [&](long long row, int slot, const RowStats& st, Pair (&z)[P][4]) {
    Pair saz = both(0.0f);
    if (!pre) return saz;
    const R* x = g.template stream<R>(kX, row, slot);
    const __nv_bfloat16* o = g.template stream<__nv_bfloat16>(kO, row, slot);
    const __nv_bfloat16* dh = g.template stream<__nv_bfloat16>(kDh, row, slot);
    const void* gr = GATE != MOE_GATE_NONE ? g.gate_row(row, slot) : nullptr;
    const Pair ay = both(p.alpha * st.r_y), ro = both(st.r_o * st.tg * st.r_y);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (V >= 8 && !cols.any(i)) continue;
      Pair q[4], f[4];
      cols.load(x, i, z[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) z[i][j] = mul2(z[i][j], ay);
      if (has_o) {
        cols.load(o, i, q);
        g.factor(0, i, f);
        if constexpr (GATE != MOE_GATE_NONE) {
          Pair gg[4];
          cols.load(gr, p.gate_f32, i, gg);
#pragma unroll
          for (int j = 0; j < 4; ++j) f[j] = mul2(f[j], gg[j]);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) z[i][j] = fma2(mul2(q[j], f[j]), ro, z[i][j]);
      }
      cols.load(dh, i, q);
      g.factor(1, i, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        aw_h[i][j] = fma2(q[j], z[i][j], aw_h[i][j]);
        saz = fma2(mul2(q[j], f[j]), z[i][j], saz);
      }
    }
    return saz;
  };
  // s, dx, S and b (in z's place; without the token gate), and this thread's
  // part of sum f s o; m: mean a z
  auto second_pass = [&](long long row, int slot, const RowStats& st, float m, Pair (&z)[P][4]) {
    const R* dy = g.template stream<R>(kDy, row, slot);
    const __nv_bfloat16* o = g.template stream<__nv_bfloat16>(kO, row, slot);
    const __nv_bfloat16* dh = g.template stream<__nv_bfloat16>(kDh, row, slot);
    const void* gr = GATE != MOE_GATE_NONE ? g.gate_row(row, slot) : nullptr;
    const Pair ro2 = both(st.r_o), rot2 = both(st.r_o * st.tg), ry2 = both(st.r_y), m2 = both(-m), alpha = both(p.alpha);
    Pair sbn = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (V >= 8 && !cols.any(i)) continue;
      Pair s[4], q[4], f[4];
      if (has_dy) {
        cols.load(dy, i, s);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = both(0.0f);
      }
      if (pre) {
        cols.load(dh, i, q);
        g.factor(1, i, f);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = fma2(ry2, fma2(z[i][j], m2, mul2(q[j], f[j])), s[j]);
      }
      if (has_dx) {
#pragma unroll
        for (int j = 0; j < 4; ++j) q[j] = mul2(alpha, s[j]);
        cols.store(static_cast<R*>(p.dx) + row * p.D, i, q);
      }
      if (!has_o) continue;
      cols.load(o, i, q);
      g.factor(0, i, f);
#pragma unroll
      for (int j = 0; j < 4; ++j) q[j] = mul2(s[j], q[j]);   // s o
      if constexpr (GATE == MOE_GATE_NONE) {
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          S[i][j] = fma2(rot2, q[j], S[i][j]);
          sbn = fma2(f[j], q[j], sbn);
          z[i][j] = mul2(s[j], f[j]);
        }
      } else {
        Pair gg[4];
        cols.load(gr, p.gate_f32, i, gg);
        if constexpr (GATE == kGateFull) {        // its gradient goes out with the row
          Pair dg[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) dg[j] = mul2(mul2(f[j], q[j]), ro2);
          cols.store(param_row(p.dgate, p.gate_f32, row * p.D), p.gate_f32, i, dg);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = mul2(f[j], gg[j]);
          S[i][j] = fma2(GATE == kGateFull ? mul2(gg[j], ro2) : ro2, q[j], S[i][j]);
          sbn = fma2(f[j], q[j], sbn);
          z[i][j] = mul2(s[j], f[j]);
        }
      }
    }
    return sbn;
  };
  // do from b; sg: sum b n = r_o sum f s o, without the token gate
  auto third_pass = [&](long long row, int slot, const RowStats& st, float sg, Pair (&z)[P][4]) {
    if (GATE == MOE_GATE_NONE && p.gate_mode == MOE_GATE_TOKEN && cols.t == 0) param_put(p.dgate, p.gate_f32, row, sg);
    const __nv_bfloat16* o = g.template stream<__nv_bfloat16>(kO, row, slot);
    const float rot = st.r_o * st.tg;
    const Pair rot2 = both(rot), mm = both(-rot * st.r_o * sg * inv_d);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (V >= 8 && !cols.any(i)) continue;
      if (post) {
        Pair q[4];
        cols.load(o, i, q);
#pragma unroll
        for (int j = 0; j < 4; ++j) z[i][j] = fma2(q[j], mm, mul2(rot2, z[i][j]));
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) z[i][j] = mul2(rot2, z[i][j]);
      }
      cols.store(p.do_ + row * p.D, i, z[i]);
    }
  };
  const bool two_sums = has_o && (post || p.gate_mode == MOE_GATE_TOKEN);

  // n rows row0, row0 + step, ...: the second pass of a row and the first of
  // the next run back to back and share one sum over the group, so that a
  // row costs one barrier; with one row in flight each has its own.
  auto rows = [&](long long row0, long long step, int n) {
    if (n <= 0) return;
    RowStats st = stats_of(row0), ahead = st;
    Pair z[P][4];
    int slot = g.template next<false>();
    Pair saz = first_pass(row0, slot, st, z);
    float m = pre ? g.sum(saz) * inv_d : 0.0f;
    for (int it = 0; it < n; ++it) {
      const long long row = row0 + it * step;
      const bool more = it + 1 < n;
      if (more) ahead = stats_of(row + step);
      const Pair sbn = second_pass(row, slot, st, m, z);
      g.release_early();
      if (p.stages > 1 && more) {
        Pair zn[P][4];
        const int slot2 = g.template next<true>();
        saz = first_pass(row + step, slot2, ahead, zn);
        float sg = 0.0f;
        g.sum_two(sbn, saz, sg, m);
        m *= inv_d;
        if (has_o) third_pass(row, slot, st, sg * st.r_o, z);
        g.release();
        slot = slot2;
#pragma unroll
        for (int i = 0; i < P; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) z[i][j] = zn[i][j];
      } else {
        const float sg = two_sums ? g.sum(sbn) : 0.0f;
        if (has_o) third_pass(row, slot, st, sg * st.r_o, z);
        g.release();
        if (more) {
          slot = g.template next<false>();
          saz = first_pass(row + step, slot, ahead, z);
          if (pre) m = g.sum(saz) * inv_d;
        }
      }
      st = ahead;
    }
  };

  if constexpr (GATE != MOE_GATE_GROUP) {
    rows(worker, workers, worker < p.T ? (p.T - 1 - worker) / workers + 1 : 0);
  } else {
    Pair aw_o[P][4];   // sum over slabs of g S
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) aw_o[i][j] = both(0.0f);
    for (long long sl = worker; sl < p.slabs; sl += workers) {
      const long long gi = sl / p.slabs_per_group, k = sl - gi * p.slabs_per_group;
      const long long r0 = gi * p.rows_per_group + p.rows_per_group * k / p.slabs_per_group;
      const int n = static_cast<int>(gi * p.rows_per_group + p.rows_per_group * (k + 1) / p.slabs_per_group - r0);
      if (V == 1) g.sync();   // the last slab's rows have been read
      g.start(r0, 1, n);
      rows(r0, 1, n);
      cp_wait<0>();
#pragma unroll
      for (int i = 0; i < P; ++i) {
        if (V >= 8 && !cols.any(i)) continue;
        Pair f[4], gg[4];
        g.factor(0, i, f);
        cols.load(param_row(p.gate, p.gate_f32, gi * p.D), p.gate_f32, i, gg);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          f[j] = mul2(f[j], S[i][j]);
          aw_o[i][j] = fma2(gg[j], S[i][j], aw_o[i][j]);
          S[i][j] = both(0.0f);
        }
        if (p.slabs_per_group == 1) cols.store(param_row(p.dgate, p.gate_f32, gi * p.D), p.gate_f32, i, f);
        else cols.store(p.gate_partial + sl * p.D, i, f);
      }
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) S[i][j] = aw_o[i][j];
  }
  cp_wait<0>();
  __syncthreads();   // the rows' memory is free: it takes the groups' sums
  float* acc = reinterpret_cast<float*>(shared + p.table);   // [D], when groups > 1
#pragma unroll
  for (int arr = 0; arr < 2; ++arr) {
    if (arr == 0 ? !has_o : !pre) continue;
    float* out = p.partial + (static_cast<long long>(arr) * gridDim.x + blockIdx.x) * p.D;
    for (int k = 0; k < p.groups; ++k) {
      if (k == g.grp) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (V >= 8 && !cols.any(i)) continue;
          Pair b[4];
          if (k > 0) cols.load(acc, i, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Pair v = arr == 0 ? S[i][j] : aw_h[i][j];
            b[j] = k > 0 ? add2(b[j], v) : v;
          }
          cols.store(k + 1 < p.groups ? acc : out, i, b);
        }
      }
      if (p.groups > 1) __syncthreads();
    }
  }
}

// The CTAs' column sums joined in a fixed order (eight interleaved sums a
// column, then those in order) and turned into the gradients: blockIdx.y = 0
// sum s n -> dw_post and a channel gate's dgate, 1 -> dw_pre.
__global__ void __launch_bounds__(256) norm_param_grad_kernel(const __grid_constant__ NormParams p, int rows,
                                                              float* dw_post, float* dw_pre) {
  __shared__ float part[8][33];
  const int a = blockIdx.y;
  if (a == 0 ? (dw_post == nullptr && p.gate_mode != MOE_GATE_CHANNEL) : dw_pre == nullptr) return;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.0f;
  if (c < p.D) {
    const float* q = p.partial + static_cast<long long>(a) * rows * p.D + c;
#pragma unroll 8
    for (int r = ry; r < rows; r += 8) s += q[static_cast<long long>(r) * p.D];
  }
  part[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < p.D) {
    for (int k = 1; k < 8; ++k) s += part[k][cx];
    if (a == 1) {
      dw_pre[c] = s;
      return;
    }
    float g = 1.0f;
    if (p.gate_mode == MOE_GATE_CHANNEL) {
      g = param_at(p.gate, p.gate_f32, c);
      const float w = p.w_post ? param_at(p.w_post, p.params_f32, c) + p.offset : 1.0f;
      param_put(p.dgate, p.gate_f32, c, w * p.beta * s);
    }
    if (dw_post) dw_post[c] = p.beta * g * s;
  }
}

// dgate[g][c] = sum of group g's slab partials, in slab order.
__global__ void __launch_bounds__(256) gate_slab_sum_kernel(const float* __restrict__ in, int per_group, int D,
                                                            void* dgate, int f32) {
  const int c = blockIdx.x * 256 + threadIdx.x;
  if (c >= D) return;
  const float* p = in + static_cast<long long>(blockIdx.y) * per_group * D + c;
  float s = 0.0f;
#pragma unroll 8
  for (int r = 0; r < per_group; ++r) s += p[static_cast<long long>(r) * D];
  param_put(dgate, f32, static_cast<long long>(blockIdx.y) * D + c, s);
}

// ------------------------------------------------------------------- host

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Shape {
  int warps, groups, stages, threads;
};

// How many groups share a CTA, and how many rows each has in flight.  As many
// groups as 16 warps and the memory hold (14 warps: backward 55 instead of 46
// us at 4096 x 4096, 80.2 and 77.8 at 16384 x 2048), in the forward no third
// one that leaves only two rows in flight (8192 x 5120: 58.3 instead of 55.7
// us); of those no more than save a round of rows (1531 x 1411 backward: four
// groups 23.3 us, five, in as many rounds, 25.8); where one round is enough, the
// forward's idle groups still help to fill the table (1 x 7168: 6.2 and 7.3 us).
Shape place(NormParams* p, bool fwd, bool vec, int sms) {
  Shape s;
  const int warp_cols = 256 * (fwd ? (vec ? kPiecesOf<8, false> : kPiecesOf<1, false>) : (vec ? kPiecesOf<8, true> : kPiecesOf<1, true>));
  s.warps = (p->D + warp_cols - 1) / warp_cols;
  p->table = (p->D * 4 + 15) / 16 * 16 * 2;
  const int room = kSharedMem - p->table;
  int most = std::max(1, std::min({kWarps / s.warps, 15, room / p->slot}));   // named barriers 1 .. 15
  if (fwd && most > 2) most = std::min(most, std::max(2, room / (3 * p->slot)));
  const int rounds = (p->T - 1) / (sms * most) + 1;
  s.groups = fwd && rounds == 1 ? most : (p->T - 1) / (sms * rounds) + 1;
  s.stages = std::max(1, std::min(4, room / (s.groups * p->slot)));
  s.threads = s.warps * s.groups * 32;
  p->warps = s.warps;
  p->groups = s.groups;
  p->stages = s.stages;
  for (Stream& q : p->in) q.piece = s.warps * 32 * 8 * q.esz;
  return s;
}

template <typename K>
cudaError_t launch(K kernel, PerDeviceOnce& once, int ctas, const Shape& s, size_t smem, const NormParams& p,
                   cudaStream_t stream) {
  const cudaError_t e =
      once.once([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedMem); });
  if (e != cudaSuccess) return e;
  kernel<<<ctas, s.threads, smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename R, int V>
cudaError_t launch_v(bool fwd, int ctas, const Shape& s, size_t smem, const NormParams& p, cudaStream_t stream) {
  static PerDeviceOnce fwd_all, forward, all, none, group, full;
  if (fwd) {
    if (p.in[kO].base && p.w_post && p.w_pre && p.y && p.gate_mode != MOE_GATE_GROUP && p.gate_mode != kGateFull)
      return launch(block_norm_fwd_kernel<R, V, true>, fwd_all, ctas, s, smem, p, stream);
    return launch(block_norm_fwd_kernel<R, V, false>, forward, ctas, s, smem, p, stream);
  }
  if (p.gate_mode == MOE_GATE_GROUP)
    return launch(block_norm_bwd_kernel<R, V, MOE_GATE_GROUP, false>, group, ctas, s, smem, p, stream);
  if (p.gate_mode == kGateFull) return launch(block_norm_bwd_kernel<R, V, kGateFull, false>, full, ctas, s, smem, p, stream);
  if (p.in[kX].base && p.in[kO].base && p.in[kDy].base && p.in[kDh].base && p.w_post && p.dx)
    return launch(block_norm_bwd_kernel<R, V, MOE_GATE_NONE, true>, all, ctas, s, smem, p, stream);
  return launch(block_norm_bwd_kernel<R, V, MOE_GATE_NONE, false>, none, ctas, s, smem, p, stream);
}

template <typename R>
cudaError_t launch_norm(bool fwd, bool vec, int ctas, const Shape& s, const NormParams& p, cudaStream_t stream) {
  const size_t rows = std::max<size_t>(static_cast<size_t>(s.groups) * s.stages * p.slot, s.groups > 1 ? 4ull * p.D : 0);
  const size_t smem = p.table + rows;
  if (!vec) return launch_v<R, 1>(fwd, ctas, s, smem, p, stream);
  return p.D % (256 * (fwd ? kPiecesOf<8, false> : kPiecesOf<8, true>)) == 0 ? launch_v<R, kFull>(fwd, ctas, s, smem, p, stream) : launch_v<R, 8>(fwd, ctas, s, smem, p, stream);
}

cudaError_t launch_norm(bool fwd, bool vec, int ctas, const Shape& s, const NormParams& p, cudaStream_t stream) {
  return p.res_f32 ? launch_norm<float>(fwd, vec, ctas, s, p, stream) : launch_norm<__nv_bfloat16>(fwd, vec, ctas, s, p, stream);
}

bool config_ok(const moe_block_norm_config* c) {
  if (!c || c->tokens < 0 || c->d_model < 1) return false;
  if (c->residual_type != MOE_TYPE_BF16 && c->residual_type != MOE_TYPE_FP32) return false;
  if (c->weight_type != MOE_TYPE_BF16 && c->weight_type != MOE_TYPE_FP32) return false;
  if (c->gate_type != MOE_TYPE_BF16 && c->gate_type != MOE_TYPE_FP32) return false;
  if (c->gate_mode < MOE_GATE_NONE || c->gate_mode > MOE_GATE_TOKEN) return false;
  if (c->gate_mode == MOE_GATE_GROUP && (c->gate_rows < 1 || c->tokens % c->gate_rows != 0)) return false;
  if (!(c->eps > 0.0f) || c->eps > 3.0e38f) return false;
  const float f[3] = {c->residual_scale, c->branch_scale, c->weight_offset};
  for (float v : f)
    if (!(v >= -3.0e38f && v <= 3.0e38f)) return false;
  return true;
}

// A row stride: 0 stands for d_model; smaller ones would overlap rows.
bool stride_ok(int64_t ld, int32_t D) { return ld == 0 || ld >= D; }

NormParams common_params(const moe_block_norm_config* c, const void* branch, const void* gate, const void* w_post,
                         const void* w_pre) {
  NormParams p{};
  p.T = c->tokens;
  p.D = c->d_model;
  p.gate = gate;
  p.w_post = w_post;
  p.w_pre = w_pre;
  p.ldy = c->y_stride ? c->y_stride : c->d_model;
  p.ldh = c->h_stride ? c->h_stride : c->d_model;
  p.gate_mode = branch ? c->gate_mode : MOE_GATE_NONE;
  p.rows_per_group = 1;
  if (p.gate_mode == MOE_GATE_GROUP) {
    p.rows_per_group = c->tokens / c->gate_rows;
    if (p.rows_per_group == 1) p.gate_mode = kGateFull;
  }
  p.params_f32 = c->weight_type == MOE_TYPE_FP32;
  p.gate_f32 = c->gate_type == MOE_TYPE_FP32;
  p.res_f32 = c->residual_type == MOE_TYPE_FP32;
  p.alpha = c->residual_scale;
  p.beta = c->branch_scale;
  p.eps = c->eps;
  p.offset = c->weight_offset;
  return p;
}

// Add a streamed tensor (stride in elements, 0: D).
void add_stream(NormParams* p, int k, const void* base, int64_t ld, moe_type type) {
  if (base == nullptr) return;
  Stream& s = p->in[k];
  s.base = static_cast<const uint8_t*>(base);
  s.esz = type == MOE_TYPE_FP32 ? 4 : 2;
  s.ld = static_cast<long long>(ld ? ld : p->D) * s.esz;
  s.row_bytes = p->D * s.esz;
  s.end = s.base + (p->T - 1) * s.ld + s.row_bytes;
}

// Choose the vector path and lay out a row's slot: with FP32 x, dy and gate at
// 8192 columns 128 KB, which fit beside the table's 64.
bool lay_out(NormParams* p) {
  bool vec = p->D % 8 == 0 && p->ldy % 8 == 0 && p->ldh % 8 == 0;
  for (const Stream& s : p->in) vec = vec && (s.base == nullptr || (s.ld / s.esz) % 8 == 0);
  p->slot = 0;
  for (Stream& s : p->in) {
    if (s.base == nullptr) continue;
    s.off = p->slot;
    p->slot += (s.row_bytes + 15) / 16 * 16 + (vec ? 0 : 16);
  }
  return vec;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_block_norm_forward(const moe_block_norm_config* cfg, const void* x, const void* branch, const void* gate,
                                  const void* post_weight, const void* pre_weight, void* y, void* h, float* stats,
                                  cudaStream_t stream) {
  if (!config_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!stride_ok(cfg->x_stride, cfg->d_model) || !stride_ok(cfg->branch_stride, cfg->d_model) ||
      !stride_ok(cfg->y_stride, cfg->d_model) || !stride_ok(cfg->h_stride, cfg->d_model))
    return MOE_ERR_INVALID_ARG;
  if (cfg->d_model > kMaxCols) return MOE_ERR_UNSUPPORTED;
  if (cfg->tokens == 0) return MOE_OK;
  if (!branch && (gate || post_weight)) return MOE_ERR_INVALID_ARG;
  if (branch && (gate != nullptr) != (cfg->gate_mode != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((pre_weight != nullptr) != (h != nullptr)) return MOE_ERR_INVALID_ARG;
  if (!x || (!y && !h)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, branch, gate, post_weight, pre_weight, static_cast<const void*>(y),
                        static_cast<const void*>(h), static_cast<const void*>(stats)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  NormParams p = common_params(cfg, branch, gate, post_weight, pre_weight);
  p.y = y;
  p.h = static_cast<__nv_bfloat16*>(h);
  p.stats = stats;
  add_stream(&p, kX, x, cfg->x_stride, cfg->residual_type);
  add_stream(&p, kO, branch, cfg->branch_stride, MOE_TYPE_BF16);
  if (p.gate_mode == kGateFull) add_stream(&p, kG, gate, 0, cfg->gate_type);
  const bool vec = lay_out(&p);
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const Shape s = place(&p, true, vec, sms);
  const int ctas = std::min(sms, p.T);
  return launch_norm(true, vec, ctas, s, p, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_block_norm_workspace_bytes(const moe_block_norm_config* cfg) {
  if (!config_ok(cfg) || cfg->d_model > kMaxCols) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  // two arrays of column sums a CTA, and (grouped gates) a row for each group of warps
  size_t rows = 2 * static_cast<size_t>(std::min(cfg->tokens, sms));
  if (cfg->gate_mode == MOE_GATE_GROUP) rows += static_cast<size_t>(std::min(cfg->tokens, 16 * sms));
  return rows * static_cast<size_t>(cfg->d_model) * sizeof(float) + 256;
}

moe_status moe_block_norm_backward(const moe_block_norm_config* cfg, const void* x, const void* branch, const void* gate,
                                   const void* post_weight, const void* pre_weight, const float* stats, const void* dy,
                                   const void* dh, void* dx, void* dbranch, void* dgate, float* dpost_weight,
                                   float* dpre_weight, void* workspace, size_t workspace_bytes, cudaStream_t stream) {
  if (!config_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (!stride_ok(cfg->x_stride, cfg->d_model) || !stride_ok(cfg->branch_stride, cfg->d_model) ||
      !stride_ok(cfg->y_stride, cfg->d_model) || !stride_ok(cfg->h_stride, cfg->d_model))
    return MOE_ERR_INVALID_ARG;
  if (cfg->d_model > kMaxCols) return MOE_ERR_UNSUPPORTED;
  const int T = cfg->tokens, D = cfg->d_model;
  if (T == 0) {   // no rows: the parameters' gradients are zero
    if (!aligned16(dgate) || !aligned16(dpost_weight) || !aligned16(dpre_weight)) return MOE_ERR_INVALID_ARG;
    auto zero = [&](void* q, size_t n) { return q ? cudaMemsetAsync(q, 0, n, stream) : cudaSuccess; };
    const size_t gsz = (cfg->gate_type == MOE_TYPE_FP32 ? 4 : 2);
    const size_t grows = cfg->gate_mode == MOE_GATE_CHANNEL ? 1 : (cfg->gate_mode == MOE_GATE_GROUP ? cfg->gate_rows : 0);
    if (zero(dpost_weight, sizeof(float) * D) != cudaSuccess || zero(dpre_weight, sizeof(float) * D) != cudaSuccess ||
        zero(grows ? dgate : nullptr, grows * D * gsz) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!branch && (gate || post_weight)) return MOE_ERR_INVALID_ARG;
  if (branch && (gate != nullptr) != (cfg->gate_mode != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((branch != nullptr) != (dbranch != nullptr)) return MOE_ERR_INVALID_ARG;
  if ((pre_weight != nullptr) != (dh != nullptr) || (!dy && !dh)) return MOE_ERR_INVALID_ARG;
  if ((post_weight != nullptr) != (dpost_weight != nullptr) || (pre_weight != nullptr) != (dpre_weight != nullptr) ||
      (gate != nullptr) != (dgate != nullptr))
    return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, branch, gate, post_weight, pre_weight, static_cast<const void*>(stats), dy, dh,
                        static_cast<const void*>(dx), static_cast<const void*>(dbranch), static_cast<const void*>(dgate),
                        static_cast<const void*>(dpost_weight), static_cast<const void*>(dpre_weight),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  if (!x || ((post_weight || pre_weight) && !stats)) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_block_norm_workspace_bytes(cfg);
  if (need == 0) return MOE_ERR_CUDA;
  if (!workspace || workspace_bytes < need) return MOE_ERR_CAPACITY;
  const int sms = device_sms();
  NormParams p = common_params(cfg, branch, gate, post_weight, pre_weight);
  p.stats = const_cast<float*>(stats);
  p.dx = dx;
  p.do_ = static_cast<__nv_bfloat16*>(dbranch);
  p.dgate = dgate;
  p.ldy = p.ldh = D;   // the outputs are contiguous
  if (pre_weight) add_stream(&p, kX, x, cfg->x_stride, cfg->residual_type);
  add_stream(&p, kO, branch, cfg->branch_stride, MOE_TYPE_BF16);
  add_stream(&p, kDy, dy, cfg->y_stride, cfg->residual_type);
  add_stream(&p, kDh, dh, cfg->h_stride, MOE_TYPE_BF16);
  if (p.gate_mode == kGateFull) add_stream(&p, kG, gate, 0, cfg->gate_type);
  const bool vec = lay_out(&p);
  const Shape s = place(&p, false, vec, sms);
  const int ctas = std::min(sms, T);
  p.partial = static_cast<float*>(workspace);
  p.gate_partial = p.partial + 2ll * ctas * D;
  if (p.gate_mode == MOE_GATE_GROUP) {
    const int per = std::max(1, std::min(ctas * s.groups / cfg->gate_rows, p.rows_per_group));
    p.slabs_per_group = per;
    p.slabs = per * cfg->gate_rows;
  }
  if (launch_norm(false, vec, ctas, s, p, stream) != cudaSuccess) return MOE_ERR_CUDA;
  if (dpost_weight || dpre_weight || p.gate_mode == MOE_GATE_CHANNEL) {
    norm_param_grad_kernel<<<dim3((D + 31) / 32, 2), 256, 0, stream>>>(p, ctas, dpost_weight, dpre_weight);
    if (cudaGetLastError() != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  if (p.gate_mode == MOE_GATE_GROUP && p.slabs_per_group > 1) {
    gate_slab_sum_kernel<<<dim3((D + 255) / 256, cfg->gate_rows), 256, 0, stream>>>(p.gate_partial, p.slabs_per_group, D,
                                                                                    dgate, p.gate_f32);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
