// Layer norm at a block boundary, with the scaled residual and dropout on the
// branch, in one pass, and its backward (moe_layer_norm_forward / _backward).
//
//   y = alpha x + beta drop(o),   m = mean y,  r = 1/sqrt(mean (y - m)^2 + eps)
//   n = (y - m) r,                h = n w + c
// h is formed from the unrounded FP32 y.  The variance is a second sum over the
// row's differences from its mean, which are in registers: no cancellation.
// Gradients, at the y that the forward wrote, with a = dh w and means over the
// row's D columns:
//   s  = dy + r (a - mean a - n mean(a n))             (gradient of y)
//   dx = alpha s,  do = beta drop(s) with the same mask,
//   dw = sum_t dh n,  dc = sum_t dh
// Reading y instead of x and o saves the backward a stream.
//
// Work layout: persistent CTAs, one per SM.  A group of W warps owns a row, P
// pieces of 8 columns a thread; as many groups share a CTA as its threads and
// shared memory hold, and take rows in turns over the CTAs.  Rows come in
// through a ring in shared memory by cp.async; a thread copies just the pieces
// it reads itself, so the copies need no barrier.
//
// Widths that 8 does not divide: row t starts t D mod 8 elements past a
// 16-byte boundary.  Each group's rows are a multiple of 8 apart, so for it
// that offset is one number: its pieces are the aligned ones, shifted by it
// against the columns, with the columns' factors shifted as well and the row's
// ends masked.  Every access stays a whole vector, the generator's groups of
// eight coincide with the pieces, and a thread's columns are the same in every
// row, so that column sums stay in registers.  A tensor whose rows start
// elsewhere (a stride that differs from D modulo 8) is read and written
// element by element in the same layout.
#include <algorithm>

#include "kernels.cuh"
#include "moe_gb300.h"
#include "philox.cuh"

namespace moe {

namespace {

constexpr int kMaxCols = 8192;
constexpr int kSharedMem = 216 * 1024;   // the columns' factors and the rows in flight
constexpr int kMaxThreads = 896;         // of a CTA: 72 registers a thread
constexpr int kMaxGroups = 15;           // named barriers 1 .. 15
constexpr int kMaxWarps = 28;

struct Stream {
  const uint8_t* base;   // NULL: not there
  long long ld;          // elements between rows
  const uint8_t* end;    // past the last row's last element
  int off;               // place in a row's slot
  int vec;               // its rows start where the layout's do, modulo 8 elements
};
// forward: x, branch; backward: y, dh, dy
enum { kX = 0, kO = 1, kY = 0, kDh = 1, kDy = 2, kStreams = 3 };

struct Out {
  void* base;            // NULL: not wanted
  long long ld;
  int vec;
};

struct LnParams {
  int T, D;
  int warps, groups, stages, slot;
  int table;             // bytes of the columns' factors
  Stream in[kStreams];
  const void* weight;    // or NULL
  const void* bias;      // forward, or NULL
  int params_f32;
  float alpha, beta, eps;
  DropParams drop;
  Out out0;              // y; dx
  Out out1;              // h; dbranch
  float* stats;          // [2][T]: mean, 1/sqrt(var + eps)
  float* partial;        // backward: [2][gridDim.x][D]: sums of dh n, dh
};

using Pair = unsigned long long;   // two FP32, one instruction (packed f32x2)
__device__ __forceinline__ Pair pair_of(float a, float b) {
  Pair r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ Pair both(float a) { return pair_of(a, a); }
__device__ __forceinline__ void split(Pair v, float& a, float& b) {
  asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v));
}
__device__ __forceinline__ Pair fma2(Pair a, Pair b, Pair c) {
  Pair r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ __forceinline__ Pair mul2(Pair a, Pair b) {
  Pair r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Pair add2(Pair a, Pair b) {
  Pair r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ float sum2(Pair v) {
  float a, b;
  split(v, a, b);
  return a + b;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ float param_at(const void* p, int f32, int i) {
  return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// 1/sqrt(x): the hardware's approximation and one Newton step.
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return r < INFINITY && r > 0.0f ? r * fmaf(-0.5f * x * r, r, 1.5f) : r;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
// the first `bytes` of 16, zeros after them
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, int bytes) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void load8(const __nv_bfloat16* p, Pair (&q)[4]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  q[0] = pair_of(bf16_lo(u.x), bf16_hi(u.x));
  q[1] = pair_of(bf16_lo(u.y), bf16_hi(u.y));
  q[2] = pair_of(bf16_lo(u.z), bf16_hi(u.z));
  q[3] = pair_of(bf16_lo(u.w), bf16_hi(u.w));
}
__device__ __forceinline__ void load8(const float* p, Pair (&q)[4]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  q[0] = pair_of(a.x, a.y);
  q[1] = pair_of(a.z, a.w);
  q[2] = pair_of(b.x, b.y);
  q[3] = pair_of(b.z, b.w);
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const Pair (&q)[4]) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) split(q[j], v[2 * j], v[2 * j + 1]);
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const Pair (&q)[4]) {
  float v[8];
#pragma unroll
  for (int j = 0; j < 4; ++j) split(q[j], v[2 * j], v[2 * j + 1]);
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// A group of warps and its rows in flight.  Pieces are numbered from the
// aligned start of a row; element j of piece c is column 8 c + j - off.
// RAGGED: D is no multiple of 8 (off may be other than 0, ends are masked).
template <typename R, int P, bool RAGGED>
struct Group {
  const LnParams& p;
  int grp, wig, nt, t, bar;
  int off, pieces;        // of its rows
  float* red;
  int turn = 0;
  uint8_t* slots;
  long long next_row, step;
  int left, fill, take;

  __device__ __forceinline__ Group(const LnParams& p_, uint8_t* shared, float (*red_all)[128]) : p(p_) {
    const int warp = threadIdx.x >> 5;
    grp = warp / p.warps;
    wig = warp - grp * p.warps;
    nt = p.warps * 32;
    t = threadIdx.x - grp * nt;
    bar = 1 + grp;
    red = red_all[grp];
    slots = shared + p.table + static_cast<size_t>(grp) * p.stages * p.slot;
    // rows blockIdx.x + a multiple of 8: the launcher makes gridDim.x one where it matters
    off = RAGGED ? static_cast<int>((static_cast<long long>(blockIdx.x) * p.D) & 7) : 0;
    pieces = RAGGED ? (p.D + off + 7) >> 3 : p.D >> 3;
  }

  __device__ __forceinline__ int piece(int i) const { return t + i * nt; }
  __device__ __forceinline__ bool any(int i) const { return piece(i) < pieces; }
  __device__ __forceinline__ bool valid(int c, int j) const {
    return static_cast<unsigned>(8 * c + j - off) < static_cast<unsigned>(p.D);
  }
  __device__ __forceinline__ bool whole(int c) const { return !RAGGED || (8 * c >= off && 8 * c + 8 <= p.D + off); }
  // zeros where the piece passes the row's ends
  __device__ __forceinline__ void mask(int c, Pair (&q)[4]) const {
    if (RAGGED && !whole(c)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a, b;
        split(q[j], a, b);
        q[j] = pair_of(valid(c, 2 * j) ? a : 0.0f, valid(c, 2 * j + 1) ? b : 0.0f);
      }
    }
  }

  __device__ __forceinline__ void sync() const {
    if (p.warps == 1) __syncwarp();
    else named_bar_sync(bar, nt);
  }

  // Sums over the group in a fixed order: an xor tree in each warp, then the
  // warps in order.  `red` holds two turns of 2 x 32 floats (zeros past the
  // warps), so one barrier a sum is enough.
  __device__ __forceinline__ float warp_sums(const float* r) const {
    const float4* q = reinterpret_cast<const float4*>(r);
    float s = (q[0].x + q[0].y) + (q[0].z + q[0].w);
    for (int k = 1; 4 * k < p.warps; ++k) s += (q[k].x + q[k].y) + (q[k].z + q[k].w);
    return s;
  }
  __device__ __forceinline__ float sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (p.warps == 1) return v;
    float* r = red + turn;
    turn ^= 64;
    if ((threadIdx.x & 31) == 0) r[wig] = v;
    named_bar_sync(bar, nt);
    return warp_sums(r);
  }
  __device__ __forceinline__ void sum_two(float& a, float& b) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      a += __shfl_xor_sync(0xFFFFFFFFu, a, o);
      b += __shfl_xor_sync(0xFFFFFFFFu, b, o);
    }
    if (p.warps == 1) return;
    float* r = red + turn;
    turn ^= 64;
    if ((threadIdx.x & 31) == 0) {
      r[wig] = a;
      r[32 + wig] = b;
    }
    named_bar_sync(bar, nt);
    a = warp_sums(r);
    b = warp_sums(r + 32);
  }

  // Send for stream k of the next row.
  template <typename X>
  __device__ __forceinline__ void copy(int k) const {
    const Stream& s = p.in[k];
    if (s.base == nullptr) return;
    X* slot = reinterpret_cast<X*>(slots + fill * p.slot + s.off);
    const X* row = reinterpret_cast<const X*>(s.base) + next_row * s.ld - off;
    if (s.vec) {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = piece(i);
        if (c >= pieces) continue;
        const uint8_t* src = reinterpret_cast<const uint8_t*>(row + 8 * c);
        const uint32_t dst = smem_u32(slot + 8 * c);
#pragma unroll
        for (int b = 0; b < 8 * static_cast<int>(sizeof(X)); b += 16) {
          if constexpr (RAGGED) {   // no byte past the tensor's last element
            const long long rest = s.end - (src + b);
            cp_async16(dst + b, rest > 0 ? src + b : s.base, rest >= 16 ? 16 : rest > 0 ? static_cast<int>(rest) : 0);
          } else {
            cp_async16(dst + b, src + b);
          }
        }
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < P; ++i) {
        const int c = piece(i);
        if (c >= pieces) continue;
#pragma unroll
        for (int j = 0; j < 8; ++j)
          if (valid(c, j)) slot[8 * c + j] = row[8 * c + j];
      }
    }
  }
  __device__ __forceinline__ void send() {
    if (left > 0) {
      copy<R>(0);
      copy<__nv_bfloat16>(1);
      copy<R>(2);
      next_row += step;
      --left;
      fill = fill + 1 == p.stages ? 0 : fill + 1;
    }
    cp_commit();
  }
  __device__ __forceinline__ void start(long long first, long long step_, int n) {
    next_row = first;
    step = step_;
    left = n;
    fill = 0;
    take = -1;
    for (int i = 0; i < p.stages; ++i) send();
  }
  // Make the next row ready: its slot.
  __device__ __forceinline__ const uint8_t* next() {
    take = take + 1 == p.stages ? 0 : take + 1;
    if (p.stages == 1) cp_wait<0>();
    else if (p.stages == 2) cp_wait<1>();
    else if (p.stages == 3) cp_wait<2>();
    else cp_wait<3>();
    return slots + take * p.slot;
  }

  // Piece c of a row of an output.
  template <typename X>
  __device__ __forceinline__ void store(const Out& o, long long row, int c, const Pair (&q)[4]) const {
    X* at = static_cast<X*>(o.base) + row * o.ld + 8 * c - off;
    if (o.vec && whole(c)) {
      store8(at, q);
    } else {
      float v[8];
#pragma unroll
      for (int j = 0; j < 4; ++j) split(q[j], v[2 * j], v[2 * j + 1]);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (valid(c, j)) put(at + j, v[j]);
    }
  }
};

// The columns' factors, one FP32 plane for each half of a piece (so that a
// warp's 16-byte reads meet no bank twice): factor `which`, half of piece c.
__device__ __forceinline__ float4* table_at(uint8_t* shared, int planes, int which, int half, int c) {
  return reinterpret_cast<float4*>(shared) + (2 * which + half) * planes + c;
}
__device__ __forceinline__ void table_load(const uint8_t* shared, int planes, int which, int c, Pair (&q)[4]) {
  const float4 a = *table_at(const_cast<uint8_t*>(shared), planes, which, 0, c);
  const float4 b = *table_at(const_cast<uint8_t*>(shared), planes, which, 1, c);
  q[0] = pair_of(a.x, a.y);
  q[1] = pair_of(a.z, a.w);
  q[2] = pair_of(b.x, b.y);
  q[3] = pair_of(b.z, b.w);
}
// Fill it (all threads; ends with a barrier).
template <int N>
__device__ __forceinline__ void make_table(const LnParams& p, uint8_t* shared, int off, int pieces, int planes) {
  for (int c = threadIdx.x; c < pieces; c += blockDim.x) {
#pragma unroll
    for (int which = 0; which < N; ++which) {
      const void* src = which ? p.bias : p.weight;
      float v[8];
      if (src && off == 0 && 8 * c + 8 <= p.D) {
        if (p.params_f32) {
          const float4 a = __ldg(static_cast<const float4*>(src) + 2 * c), b = __ldg(static_cast<const float4*>(src) + 2 * c + 1);
          v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
          const uint4 u = __ldg(static_cast<const uint4*>(src) + c);
          v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
          v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
        }
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int d = 8 * c + j - off;
          v[j] = d < 0 || d >= p.D ? 0.0f : src ? param_at(src, p.params_f32, d) : which ? 0.0f : 1.0f;
        }
      }
      *table_at(shared, planes, which, 0, c) = make_float4(v[0], v[1], v[2], v[3]);
      *table_at(shared, planes, which, 1, c) = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
  __syncthreads();
}

// q *= f where kept, 0 elsewhere.
__device__ __forceinline__ void drop_scale(const PhiloxKey& key, const DropParams& d, unsigned long long group, float f,
                                           Pair (&q)[4]) {
  const uint4 w = philox(key, group);
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    float a, b;
    split(q[j], a, b);
    q[j] = pair_of(kept(w, 2 * j, d.threshold) ? a * f : 0.0f, kept(w, 2 * j + 1, d.threshold) ? b * f : 0.0f);
  }
}

template <typename R, int P, bool RAGGED, bool DROP>
__global__ void __launch_bounds__(kMaxThreads, 1) layer_norm_fwd_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) float red_all[kMaxGroups][128];
  Group<R, P, RAGGED> g(p, shared, red_all);
  const int planes = (p.D + 7 + (RAGGED ? 7 : 0)) >> 3;
  const int first = g.grp * gridDim.x + blockIdx.x, step = gridDim.x * p.groups;
  const int n = first < p.T ? (p.T - 1 - first) / step + 1 : 0;
  for (int i = threadIdx.x; i < kMaxGroups * 128; i += blockDim.x) (&red_all[0][0])[i] = 0.0f;
  g.start(first, step, n);
  PhiloxKey key{};
  if (DROP) key = philox_key(p.drop);
  make_table<2>(p, shared, g.off, g.pieces, planes);
  const bool has_o = p.in[kO].base != nullptr;
  const float inv_d = 1.0f / static_cast<float>(p.D), beta = p.beta * p.drop.scale;
  long long row = first;
  for (int it = 0; it < n; ++it, row += step) {
    const uint8_t* slot = g.next();
    const unsigned long long group0 = DROP ? static_cast<unsigned long long>(row * p.D) >> 3 : 0;
    Pair y[P][4], s = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
      load8(reinterpret_cast<const R*>(slot + p.in[kX].off) + 8 * c, y[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i][j] = mul2(y[i][j], both(p.alpha));
      if (has_o) {
        Pair o[4];
        load8(reinterpret_cast<const __nv_bfloat16*>(slot + p.in[kO].off) + 8 * c, o);
        if constexpr (DROP) {
          drop_scale(key, p.drop, group0 + c, beta, o);
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i][j] = add2(y[i][j], o[j]);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) y[i][j] = fma2(o[j], both(beta), y[i][j]);
        }
      }
      g.mask(c, y[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s = add2(s, y[i][j]);
      if (p.out0.base) g.template store<R>(p.out0, row, c, y[i]);
    }
    g.send();
    const float mean = g.sum(sum2(s)) * inv_d;
    s = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i][j] = add2(y[i][j], both(-mean));
      g.mask(c, y[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fma2(y[i][j], y[i][j], s);
    }
    const float r = inv_sqrt(fmaf(g.sum(sum2(s)), inv_d, p.eps));
    if (p.stats && g.t == 0) {
      p.stats[row] = mean;
      p.stats[p.T + row] = r;
    }
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
      Pair w[4], b[4];
      table_load(shared, planes, 0, c, w);
      table_load(shared, planes, 1, c, b);
#pragma unroll
      for (int j = 0; j < 4; ++j) w[j] = fma2(mul2(y[i][j], both(r)), w[j], b[j]);
      g.template store<__nv_bfloat16>(p.out1, row, c, w);
    }
  }
  cp_wait<0>();
}

template <typename R, int P, bool RAGGED, bool DROP>
__global__ void __launch_bounds__(kMaxThreads, 1) layer_norm_bwd_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) float red_all[kMaxGroups][128];
  Group<R, P, RAGGED> g(p, shared, red_all);
  const int planes = (p.D + 7 + (RAGGED ? 7 : 0)) >> 3;
  const int first = g.grp * gridDim.x + blockIdx.x, step = gridDim.x * p.groups;
  const int n = first < p.T ? (p.T - 1 - first) / step + 1 : 0;
  for (int i = threadIdx.x; i < kMaxGroups * 128; i += blockDim.x) (&red_all[0][0])[i] = 0.0f;
  g.start(first, step, n);
  PhiloxKey key{};
  if (DROP) key = philox_key(p.drop);
  make_table<1>(p, shared, g.off, g.pieces, planes);
  const bool has_dy = p.in[kDy].base != nullptr;
  const float inv_d = 1.0f / static_cast<float>(p.D), beta = p.beta * p.drop.scale;
  Pair sw[P][4], sb[P][4];   // sums over the group's rows of dh n and dh
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sw[i][j] = sb[i][j] = both(0.0f);
  long long row = first;
  float mean = 0.0f, r = 0.0f;
  if (n > 0) {
    mean = p.stats[row];
    r = p.stats[p.T + row];
  }
  for (int it = 0; it < n; ++it, row += step) {
    const uint8_t* slot = g.next();
    const R* ys = reinterpret_cast<const R*>(slot + p.in[kY].off);
    const __nv_bfloat16* hs = reinterpret_cast<const __nv_bfloat16*>(slot + p.in[kDh].off);
    float mean1 = 0.0f, r1 = 0.0f;   // the next row's
    if (it + 1 < n) {
      mean1 = p.stats[row + step];
      r1 = p.stats[p.T + row + step];
    }
    const Pair r2 = both(r), mr = both(-mean * r);
    Pair sa = both(0.0f), san = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
      Pair n2[4], dh[4], w[4];
      load8(ys + 8 * c, n2);
      load8(hs + 8 * c, dh);
      g.mask(c, n2);
      g.mask(c, dh);
      table_load(shared, planes, 0, c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n2[j] = fma2(n2[j], r2, mr);
        sb[i][j] = add2(sb[i][j], dh[j]);
        sw[i][j] = fma2(dh[j], n2[j], sw[i][j]);
        dh[j] = mul2(dh[j], w[j]);
        sa = add2(sa, dh[j]);
        san = fma2(dh[j], n2[j], san);
      }
    }
    float ma = sum2(sa), man = sum2(san);
    g.sum_two(ma, man);
    const Pair rma = both(-r * ma * inv_d), rman = both(-r * man * inv_d);
    const unsigned long long group0 = DROP ? static_cast<unsigned long long>(row * p.D) >> 3 : 0;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
      Pair n2[4], dh[4], w[4], s[4];
      load8(ys + 8 * c, n2);
      load8(hs + 8 * c, dh);
      table_load(shared, planes, 0, c, w);
      if (has_dy) {
        load8(reinterpret_cast<const R*>(slot + p.in[kDy].off) + 8 * c, s);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = both(0.0f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n2[j] = fma2(n2[j], r2, mr);
        s[j] = add2(s[j], fma2(n2[j], rman, fma2(mul2(dh[j], w[j]), r2, rma)));
        n2[j] = mul2(s[j], both(p.alpha));
      }
      if (p.out0.base) g.template store<R>(p.out0, row, c, n2);
      if (p.out1.base) {
        if constexpr (DROP) {
          drop_scale(key, p.drop, group0 + c, beta, s);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) s[j] = mul2(s[j], both(beta));
        }
        g.template store<__nv_bfloat16>(p.out1, row, c, s);
      }
    }
    g.send();
    mean = mean1;
    r = r1;
  }
  cp_wait<0>();
  __syncthreads();   // the rows' memory is free: it takes the groups' sums
  float4* acc = reinterpret_cast<float4*>(shared + p.table);   // [2 halves][planes], when groups > 1
#pragma unroll
  for (int arr = 0; arr < 2; ++arr) {
    float* out = p.partial + (static_cast<long long>(arr) * gridDim.x + blockIdx.x) * p.D;
    for (int k = 0; k < p.groups; ++k) {
      if (k == g.grp) {
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c = g.piece(i);
          if (c >= g.pieces) continue;
          Pair b[4];
          if (k > 0) table_load(reinterpret_cast<uint8_t*>(acc), planes, 0, c, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Pair v = arr == 0 ? sw[i][j] : sb[i][j];
            b[j] = k > 0 ? add2(b[j], v) : v;
          }
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) split(b[j], v[2 * j], v[2 * j + 1]);
          if (k + 1 < p.groups) {
            acc[c] = make_float4(v[0], v[1], v[2], v[3]);
            acc[planes + c] = make_float4(v[4], v[5], v[6], v[7]);
          } else {
#pragma unroll
            for (int j = 0; j < 8; ++j)
              if (!RAGGED || g.valid(c, j)) out[8 * c + j - g.off] = v[j];
          }
        }
      }
      if (p.groups > 1) __syncthreads();
    }
  }
}

// The CTAs' column sums joined in a fixed order (eight interleaved sums a
// column, then those in order): blockIdx.y = 0 dweight, 1 dbias.
__global__ void __launch_bounds__(256) layer_norm_sums_kernel(const float* partial, int rows, int D, float* dweight,
                                                              float* dbias) {
  __shared__ float part[8][33];
  float* out = blockIdx.y ? dbias : dweight;
  if (out == nullptr) return;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.0f;
  if (c < D) {
    const float* q = partial + static_cast<long long>(blockIdx.y) * rows * D + c;
#pragma unroll 8
    for (int r = ry; r < rows; r += 8) s += q[static_cast<long long>(r) * D];
  }
  part[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < D) {
    for (int k = 1; k < 8; ++k) s += part[k][cx];
    out[c] = s;
  }
}

// ------------------------------------------------------------------- host

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }
bool finite(float v) { return v >= -3.0e38f && v <= 3.0e38f; }

bool config_ok(const moe_layer_norm_config* c) {
  if (!c || c->tokens < 0 || c->d_model < 1) return false;
  if (c->residual_type != MOE_TYPE_BF16 && c->residual_type != MOE_TYPE_FP32) return false;
  if (c->weight_type != MOE_TYPE_BF16 && c->weight_type != MOE_TYPE_FP32) return false;
  if (!(c->eps > 0.0f) || c->eps > 3.0e38f) return false;
  if (!finite(c->residual_scale) || !finite(c->branch_scale)) return false;
  if (!(c->dropout >= 0.0 && c->dropout <= 1.0)) return false;
  for (int64_t ld : {c->x_stride, c->branch_stride, c->y_stride, c->h_stride})
    if (ld != 0 && ld < c->d_model) return false;
  return true;
}

LnParams common_params(const moe_layer_norm_config* c) {
  LnParams p{};
  p.T = c->tokens;
  p.D = c->d_model;
  p.params_f32 = c->weight_type == MOE_TYPE_FP32;
  p.alpha = c->residual_scale;
  p.beta = c->branch_scale;
  p.eps = c->eps;
  return p;
}

// Rows whose stride is D's modulo 8 start where the layout's pieces do.
int phased(long long ld, const LnParams& p) { return (ld - p.D) % 8 == 0 || p.T == 1; }

void add_stream(LnParams* p, int k, const void* base, int64_t ld, int esz) {
  if (base == nullptr) return;
  Stream& s = p->in[k];
  s.base = static_cast<const uint8_t*>(base);
  s.ld = ld ? ld : p->D;
  s.end = s.base + ((p->T - 1) * s.ld + p->D) * esz;
  s.vec = phased(s.ld, *p);
  s.off = p->slot;
  p->slot += (p->D + 14) / 8 * 8 * esz;
}
Out make_out(const LnParams& p, void* base, int64_t ld) {
  const long long l = ld ? ld : p.D;
  return {base, l, phased(l, p)};
}

struct Shape {
  int pieces, ctas, threads;
  size_t smem;
};

// Pieces a thread, warps a row, groups a CTA and rows in flight.
bool place(LnParams* p, bool fwd, int sms, Shape* s) {
  const bool ragged = p->D % 8 != 0;
  const int all = (p->D + 7 + (ragged ? 7 : 0)) / 8;   // pieces of a row
  // the largest number of pieces a thread that wastes no more than a sixth of the lanes
  const int most = fwd ? 4 : 2;
  s->pieces = 1;
  for (int q = 2; q <= most; q *= 2)
    if ((all + 32 * q - 1) / (32 * q) * (32 * q) * 6 <= all * 7) s->pieces = q;
  if ((all + 32 * s->pieces - 1) / (32 * s->pieces) > kMaxWarps) s->pieces *= 2;
  p->warps = (all + 32 * s->pieces - 1) / (32 * s->pieces);
  p->table = (fwd ? 2 : 1) * all * 32;
  const int room = kSharedMem - p->table;
  int groups = std::max(1, std::min({kMaxWarps / p->warps, kMaxGroups, room / (2 * p->slot)}));
  groups = std::min(groups, (p->T - 1) / sms + 1);
  p->groups = groups;
  p->stages = std::max(1, std::min(4, room / (groups * p->slot)));
  if (p->stages * p->slot > room) return false;
  s->threads = p->warps * groups * 32;
  // a group's rows have to be a multiple of 8 apart
  const int ctas = std::min(sms, p->T);
  s->ctas = !ragged || p->T <= sms ? ctas : std::max(8, sms / 8 * 8);
  const size_t rows = std::max<size_t>(static_cast<size_t>(groups) * p->stages * p->slot, groups > 1 ? all * 32ull : 0);
  s->smem = p->table + rows;
  return true;
}

template <typename K>
cudaError_t launch(K kernel, PerDeviceOnce& once, const Shape& s, const LnParams& p, cudaStream_t stream) {
  const cudaError_t e =
      once.once([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSharedMem); });
  if (e != cudaSuccess) return e;
  kernel<<<s.ctas, s.threads, s.smem, stream>>>(p);
  return cudaGetLastError();
}

template <typename R, int P, bool RAGGED, bool DROP>
cudaError_t launch_as(bool fwd, const Shape& s, const LnParams& p, cudaStream_t stream) {
  static PerDeviceOnce f, b;
  if (fwd) return launch(layer_norm_fwd_kernel<R, P, RAGGED, DROP>, f, s, p, stream);
  if constexpr (P <= 2) return launch(layer_norm_bwd_kernel<R, P, RAGGED, DROP>, b, s, p, stream);
  else return cudaErrorInvalidConfiguration;
}
template <typename R, int P>
cudaError_t launch_p(bool fwd, const Shape& s, const LnParams& p, cudaStream_t stream) {
  const bool ragged = p.D % 8 != 0, drop = p.drop.rng != nullptr;
  if (ragged) return drop ? launch_as<R, P, true, true>(fwd, s, p, stream) : launch_as<R, P, true, false>(fwd, s, p, stream);
  return drop ? launch_as<R, P, false, true>(fwd, s, p, stream) : launch_as<R, P, false, false>(fwd, s, p, stream);
}
template <typename R>
cudaError_t launch_r(bool fwd, const Shape& s, const LnParams& p, cudaStream_t stream) {
  if (s.pieces == 1) return launch_p<R, 1>(fwd, s, p, stream);
  if (s.pieces == 2) return launch_p<R, 2>(fwd, s, p, stream);
  return launch_p<R, 4>(fwd, s, p, stream);
}
cudaError_t launch_norm(bool fwd, bool f32, const Shape& s, const LnParams& p, cudaStream_t stream) {
  return f32 ? launch_r<float>(fwd, s, p, stream) : launch_r<__nv_bfloat16>(fwd, s, p, stream);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_layer_norm_forward(const moe_layer_norm_config* cfg, const void* x, const void* branch, const void* weight,
                                  const void* bias, const int64_t* rng, void* y, void* h, float* stats,
                                  cudaStream_t stream) {
  if (!config_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (cfg->d_model > kMaxCols) return MOE_ERR_UNSUPPORTED;
  if (cfg->tokens == 0) return MOE_OK;
  if (!x || !h) return MOE_ERR_INVALID_ARG;
  LnParams p = common_params(cfg);
  if (!drop_params(&p.drop, rng, cfg->dropout, cfg->site)) return MOE_ERR_INVALID_ARG;
  if (p.drop.threshold && (!rng || !branch)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, branch, weight, bias, static_cast<const void*>(rng), static_cast<const void*>(y),
                        static_cast<const void*>(h), static_cast<const void*>(stats)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  const bool f32 = cfg->residual_type == MOE_TYPE_FP32;
  p.weight = weight;
  p.bias = bias;
  p.stats = stats;
  add_stream(&p, kX, x, cfg->x_stride, f32 ? 4 : 2);
  add_stream(&p, kO, branch, cfg->branch_stride, 2);
  p.out0 = make_out(p, y, cfg->y_stride);
  p.out1 = make_out(p, h, cfg->h_stride);
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  Shape s;
  if (!place(&p, true, sms, &s)) return MOE_ERR_UNSUPPORTED;
  return launch_norm(true, f32, s, p, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_layer_norm_workspace_bytes(const moe_layer_norm_config* cfg) {
  if (!config_ok(cfg) || cfg->d_model > kMaxCols) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  // two arrays of column sums a CTA
  return 2 * static_cast<size_t>(std::min(cfg->tokens, std::max(8, sms))) * cfg->d_model * sizeof(float) + 256;
}

moe_status moe_layer_norm_backward(const moe_layer_norm_config* cfg, const void* y, const void* weight, const float* stats,
                                   const int64_t* rng, const void* dy, const void* dh, void* dx, void* dbranch,
                                   float* dweight, float* dbias, void* workspace, size_t workspace_bytes,
                                   cudaStream_t stream) {
  if (!config_ok(cfg)) return MOE_ERR_INVALID_ARG;
  if (cfg->d_model > kMaxCols) return MOE_ERR_UNSUPPORTED;
  const int T = cfg->tokens, D = cfg->d_model;
  if (T == 0) {   // no rows: the parameters' gradients are zero
    if (!aligned16(dweight) || !aligned16(dbias)) return MOE_ERR_INVALID_ARG;
    auto zero = [&](void* q) { return q ? cudaMemsetAsync(q, 0, sizeof(float) * D, stream) : cudaSuccess; };
    return zero(dweight) == cudaSuccess && zero(dbias) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
  }
  if (!y || !stats || !dh || (!dx && !dbranch && !dweight && !dbias)) return MOE_ERR_INVALID_ARG;
  LnParams p = common_params(cfg);
  if (!drop_params(&p.drop, rng, cfg->dropout, cfg->site)) return MOE_ERR_INVALID_ARG;
  if (p.drop.threshold && (!rng || !dbranch)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {y, weight, static_cast<const void*>(stats), static_cast<const void*>(rng), dy, dh,
                        static_cast<const void*>(dx), static_cast<const void*>(dbranch),
                        static_cast<const void*>(dweight), static_cast<const void*>(dbias),
                        static_cast<const void*>(workspace)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_layer_norm_workspace_bytes(cfg);
  if (need == 0) return MOE_ERR_CUDA;
  if (!workspace || workspace_bytes < need) return MOE_ERR_CAPACITY;
  const int sms = device_sms();
  const bool f32 = cfg->residual_type == MOE_TYPE_FP32;
  p.weight = weight;
  p.stats = const_cast<float*>(stats);
  p.partial = static_cast<float*>(workspace);
  add_stream(&p, kY, y, cfg->x_stride, f32 ? 4 : 2);
  add_stream(&p, kDh, dh, cfg->h_stride, 2);
  add_stream(&p, kDy, dy, cfg->y_stride, f32 ? 4 : 2);
  p.out0 = make_out(p, dx, 0);
  p.out1 = make_out(p, dbranch, 0);
  Shape s;
  if (!place(&p, false, sms, &s)) return MOE_ERR_UNSUPPORTED;
  if (launch_norm(false, f32, s, p, stream) != cudaSuccess) return MOE_ERR_CUDA;
  if (dweight || dbias) {
    layer_norm_sums_kernel<<<dim3((D + 31) / 32, 2), 256, 0, stream>>>(p.partial, s.ctas, D, dweight, dbias);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
