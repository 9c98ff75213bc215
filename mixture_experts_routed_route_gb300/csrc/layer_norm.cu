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
// pieces of 8 columns a thread; as many groups share a CTA as its threads hold,
// and take rows in turns over the CTAs.  The forward keeps a row in registers
// from its one read to its results, and sends for the next row as soon as the
// row's own values have been used.  The backward, whose registers hold the
// column sums, has its rows in flight in a ring in shared memory (cp.async; a
// thread copies the pieces it reads itself, so the copies need no barrier).
// Dropout's mask of the next row is drawn while that row is under way; where a
// wide row's group leaves warps of its CTA over, by those.
//
// What bounds it (BF16 with a branch, one GB300): the stream.  Forward 2048 x 7168
// 21.4 us (5.5 TB/s; floor 17.3), 8192 x 7168 76 us (6.2 TB/s); the backward with
// its second kernel 34.3 us (floor 21.6) and 100.5 us (5.8 TB/s).  Short inputs
// add a fixed part (launch, first row, last stores; the backward's column sums
// and second kernel, 12 us).  With dropout: forward 26.3 and 92 us, backward 36.5
// and 112 us.  The generator's products alone would be under 4 us of 2048 x 7168
// (4 cycles a warp and scheduler each), and half of the issue slots are idle: it
// is that a row's mask and sums stand between two barriers, one row a CTA at a
// time.  Odd widths: 16384 x 1411 forward 37 us, with dropout 56, backward 54 and
// 72 (16384 x 1408: forward 31 and 37.6, backward 42.8).  Odd widths above 8185
// take four pieces a thread and spill: 4096 x 8191 forward 93 and 102 us, backward
// 194 and 227 (4096 x 8184: 57 and 69, 73 and 89).
// Tried and slower: forward rows through a ring too (27.5 us, 88.7 us), 24 warps
// (80 registers: one row in flight a CTA, 24.7 us), one piece a thread (25.6 us);
// backward with rows in registers (56 us, spills), 28 warps without a row's
// normalised values kept (53.7 us), column sums that leave element by element
// (39.2 us); masks drawn apart for two groups in the forward, which leaves
// 64 registers (28.9 us), with two or three rows in flight (27.2, 28.8 us), in the
// backward as finished words instead of raw numbers, or for half of a row (40.3
// and 42.5 us).
//
// Widths that 8 does not divide: row t starts t D mod 8 elements past a
// 16-byte boundary.  Each group's rows are a multiple of 8 apart, so for it
// that offset is one number: its pieces are the aligned ones, shifted by it
// against the columns, with the columns' factors shifted as well and the row's
// ends masked.  Every access but at the ends stays a whole vector, the
// generator's groups of eight coincide with the pieces, and a thread's columns
// are the same in every row, so that column sums stay in registers.  A tensor
// whose rows start elsewhere (a stride that differs from D modulo 8) is read
// and written element by element in the same layout.
#include <algorithm>

#include "kernels.cuh"
#include "moe_gb300.h"
#include "philox.cuh"

namespace moe {

namespace {

constexpr int kMaxCols = 8192;
// Threads of a CTA: 896 have 72 registers each, 512 have 128.  Odd widths with
// dropout run out of the 72 (16384 x 1411 with 896 threads 64 us, with 512 57; FP32 75 and 63;
// without dropout 38 and 42).
constexpr int fwd_threads(bool odd, bool drop) { return odd && drop ? 512 : 896; }
constexpr int kBwdThreads = 512;   // 128 registers: the column sums and a row's normalised values stay in them
constexpr int kMaxGroups = 15;     // named barriers 1 .. 15
constexpr int kSecondBarrier = 8;  // of one group's second sum, where it shares that with the warps that draw

struct Tensor {
  void* base;      // NULL: not there
  long long ld;    // elements between rows
  int vec;         // its rows start where the layout's do, modulo 8 elements
  const uint8_t* end;   // past its last element
};

struct LnParams {
  int T, D;
  int warps, groups;
  int stages, slot;      // backward: rows in flight per group, bytes of one
  int drawers;           // warps that draw the masks of the others' rows
  int masks;             // where these are in shared memory, in bytes
  Tensor x, o, dy, dh;   // forward: x, branch; backward: x is y
  Tensor out0;           // y; dx
  Tensor out1;           // h; dbranch
  const void* weight;    // or NULL
  const void* bias;      // forward, or NULL
  int params_f32;
  float alpha, beta, eps;
  DropParams drop;
  float* stats;          // [2][T]: mean, 1/sqrt(var + eps)
  float* partial;        // backward: [2][gridDim.x][pieces of 8]: sums of dh n, dh
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

__device__ __forceinline__ float param_at(const void* p, int f32, int i) {
  return f32 ? static_cast<const float*>(p)[i] : __bfloat162float(static_cast<const __nv_bfloat16*>(p)[i]);
}

// 1/sqrt(x): the hardware's approximation and one Newton step.
__device__ __forceinline__ float inv_sqrt(float x) {
  const float r = rsqrtf(x);
  return r < INFINITY && r > 0.0f ? r * fmaf(-0.5f * x * r, r, 1.5f) : r;
}

// Eight elements as they lie in memory.
template <typename X>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void set(const Pair (&q)[4]) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 4; ++j) split(q[j], v[2 * j], v[2 * j + 1]);
    u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  // element by element, those of the bits `on`; zeros elsewhere
  __device__ __forceinline__ void gather(const __nv_bfloat16* p, uint32_t on) {
    uint32_t v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = on >> j & 1 ? reinterpret_cast<const unsigned short*>(p)[j] : 0;
    u = make_uint4(v[0] | v[1] << 16, v[2] | v[3] << 16, v[4] | v[5] << 16, v[6] | v[7] << 16);
  }
  __device__ __forceinline__ void only(uint32_t on) {   // zeros elsewhere
    uint32_t* w[4] = {&u.x, &u.y, &u.z, &u.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
      *w[j] &= (on >> (2 * j) & 1 ? 0x0000FFFFu : 0u) | (on >> (2 * j) & 2 ? 0xFFFF0000u : 0u);
  }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  // Elements lo .. hi - 1 of a piece at a row's end.  vec: the piece is aligned; what is missing then is at
  // one of its ends, and one, two and four elements at a time are enough.
  __device__ __forceinline__ void store(__nv_bfloat16* p, int lo, int hi, bool vec) const {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    unsigned short* s = reinterpret_cast<unsigned short*>(p);
    if (vec && hi == 8) {
      const int i = (lo + 1) & 6;   // the first whole pair (8 & 6 = 0: none)
      if (lo & 1) s[lo] = static_cast<unsigned short>((lo < 4 ? (lo == 1 ? w[0] : w[1]) : lo == 5 ? w[2] : w[3]) >> 16);
      if (i & 2) *reinterpret_cast<uint32_t*>(s + i) = i == 2 ? w[1] : w[3];
      if (lo <= 4) *reinterpret_cast<uint2*>(s + 4) = make_uint2(w[2], w[3]);
    } else if (vec && lo == 0) {
      if (hi & 4) *reinterpret_cast<uint2*>(s) = make_uint2(w[0], w[1]);
      if (hi & 2) *reinterpret_cast<uint32_t*>(s + (hi & 4)) = hi & 4 ? w[2] : w[0];
      if (hi & 1) s[hi - 1] = static_cast<unsigned short>(hi < 4 ? (hi == 1 ? w[0] : w[1]) : hi == 5 ? w[2] : w[3]);
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= lo && j < hi) s[j] = static_cast<unsigned short>(w[j >> 1] >> (16 * (j & 1)));
    }
  }
  __device__ __forceinline__ void keep(const uint4& m) { u = make_uint4(u.x & m.x, u.y & m.y, u.z & m.z, u.w & m.w); }
  __device__ __forceinline__ void get(Pair (&q)[4]) const {
    q[0] = pair_of(bf16_lo(u.x), bf16_hi(u.x));
    q[1] = pair_of(bf16_lo(u.y), bf16_hi(u.y));
    q[2] = pair_of(bf16_lo(u.z), bf16_hi(u.z));
    q[3] = pair_of(bf16_lo(u.w), bf16_hi(u.w));
  }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void set(const Pair (&q)[4]) {
    split(q[0], a.x, a.y);
    split(q[1], a.z, a.w);
    split(q[2], b.x, b.y);
    split(q[3], b.z, b.w);
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void store(float* p, int lo, int hi, bool vec) const {
    const float v[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (vec && hi == 8) {
      const int i = (lo + 1) & 6;
      if (lo & 1) p[lo] = lo < 4 ? (lo == 1 ? v[1] : v[3]) : lo == 5 ? v[5] : v[7];
      if (i & 2) *reinterpret_cast<float2*>(p + i) = i == 2 ? make_float2(v[2], v[3]) : make_float2(v[6], v[7]);
      if (lo <= 4) *reinterpret_cast<float4*>(p + 4) = b;
    } else if (vec && lo == 0) {
      if (hi & 4) *reinterpret_cast<float4*>(p) = a;
      if (hi & 2) *reinterpret_cast<float2*>(p + (hi & 4)) = hi & 4 ? make_float2(v[4], v[5]) : make_float2(v[0], v[1]);
      if (hi & 1) p[hi - 1] = hi < 4 ? (hi == 1 ? v[0] : v[2]) : hi == 5 ? v[4] : v[6];
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j >= lo && j < hi) p[j] = v[j];
    }
  }
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void gather(const float* p, uint32_t on) {
    float v[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = on >> j & 1 ? p[j] : 0.0f;
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void only(uint32_t on) {
    float* w[8] = {&a.x, &a.y, &a.z, &a.w, &b.x, &b.y, &b.z, &b.w};
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!(on >> j & 1)) *w[j] = 0.0f;
  }
  __device__ __forceinline__ void get(Pair (&q)[4]) const {
    q[0] = pair_of(a.x, a.y);
    q[1] = pair_of(a.z, a.w);
    q[2] = pair_of(b.x, b.y);
    q[3] = pair_of(b.z, b.w);
  }
};

// What is read where a row's vectors may not be.
__device__ uint4 g_zeros[2];

// A group of warps.  Pieces are numbered from the aligned start of a row;
// element j of piece c is column 8 c + j - off.  ODD: D is no multiple of 8 (off
// may be other than 0, ends are masked), or a tensor's rows start elsewhere.
template <int P, bool ODD>
struct Group {
  const LnParams& p;
  int grp, wig, nt, t, bar;
  int members;            // threads that meet at the barrier of sum_two
  int off, pieces;        // of its rows
  float* red;
  int turn = 0;

  __device__ __forceinline__ Group(const LnParams& p_, float (*red_all)[128]) : p(p_) {
    const int warp = threadIdx.x >> 5;
    grp = warp / p.warps;
    wig = warp - grp * p.warps;
    nt = members = p.warps * 32;
    t = threadIdx.x - grp * nt;
    bar = 1 + grp;
    red = red_all[grp];
    // rows blockIdx.x + a multiple of 8: the launcher makes gridDim.x one where it matters
    off = ODD ? static_cast<int>((static_cast<long long>(blockIdx.x) * p.D) & 7) : 0;
    pieces = ODD ? (p.D + off + 7) >> 3 : p.D >> 3;
    for (int i = threadIdx.x; i < kMaxGroups * 128; i += blockDim.x) (&red_all[0][0])[i] = 0.0f;
  }

  __device__ __forceinline__ int piece(int i) const { return t + i * nt; }
  __device__ __forceinline__ bool valid(int c, int j) const {
    return static_cast<unsigned>(8 * c + j - off) < static_cast<unsigned>(p.D);
  }
  __device__ __forceinline__ bool whole(int c) const { return !ODD || (8 * c >= off && 8 * c + 8 <= p.D + off); }
  // Its columns of the row, a bit each.
  __device__ __forceinline__ uint32_t columns(int c) const {
    const int lo = max(0, off - 8 * c), hi = max(0, min(8, p.D + off - 8 * c));
    return (0xFFu << lo) & (0xFFu >> (8 - hi));
  }
  // zeros where the piece passes the row's ends
  __device__ __forceinline__ void mask(int c, Pair (&q)[4]) const {
    if (ODD && !whole(c)) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        float a, b;
        split(q[j], a, b);
        q[j] = pair_of(valid(c, 2 * j) ? a : 0.0f, valid(c, 2 * j + 1) ? b : 0.0f);
      }
    }
  }

  // Sums over the group in a fixed order: an xor tree in each warp, then a tree
  // over the warps.  `count` threads meet at the barrier `id`.
  // `red` holds two turns of 2 x 32 floats (zeros past the warps), so one barrier
  // a sum is enough.
  __device__ __forceinline__ float warp_sums(const float* r) const {
    const float4* q = reinterpret_cast<const float4*>(r);
    float s = (q[0].x + q[0].y) + (q[0].z + q[0].w);
    if (p.warps > 4) s += (q[1].x + q[1].y) + (q[1].z + q[1].w);
    if (p.warps > 8) s += ((q[2].x + q[2].y) + (q[2].z + q[2].w)) + ((q[3].x + q[3].y) + (q[3].z + q[3].w));
    if (p.warps > 16)
      s += (((q[4].x + q[4].y) + (q[4].z + q[4].w)) + ((q[5].x + q[5].y) + (q[5].z + q[5].w))) +
           (((q[6].x + q[6].y) + (q[6].z + q[6].w)) + ((q[7].x + q[7].y) + (q[7].z + q[7].w)));
    return s;
  }
  __device__ __forceinline__ float sum(float v, int id, int count) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (p.warps == 1) return v;
    float* r = red + turn;
    turn ^= 64;
    if ((threadIdx.x & 31) == 0) r[wig] = v;
    named_bar_sync(id, count);
    return warp_sums(r);
  }
  __device__ __forceinline__ float sum(float v) { return sum(v, bar, nt); }
  // Two at once: the lower half of a warp carries a, the upper half b.
  __device__ __forceinline__ void sum_two(float& a, float& b) {
    const bool upper = threadIdx.x & 16;
    float v = (upper ? b : a) + __shfl_xor_sync(0xFFFFFFFFu, upper ? a : b, 16);
#pragma unroll
    for (int o = 8; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    if (p.warps == 1) {
      a = __shfl_sync(0xFFFFFFFFu, v, 0);
      b = __shfl_sync(0xFFFFFFFFu, v, 16);
      return;
    }
    float* r = red + turn;
    turn ^= 64;
    if ((threadIdx.x & 15) == 0) r[2 * (threadIdx.x & 16) + wig] = v;
    named_bar_sync(bar, members);
    a = warp_sums(r);
    b = warp_sums(r + 32);
  }

  // Whether whole vectors may be read along the row: those at its ends hold
  // elements of the rows beside it, but none past the tensor's end.
  template <typename X>
  __device__ __forceinline__ bool vectors(const Tensor& s, long long row) const {
    const X* end = static_cast<const X*>(s.base) + row * s.ld - off + 8 * pieces;
    return !ODD || (s.vec && reinterpret_cast<const uint8_t*>(end) <= s.end);
  }
  // Piece c, at src, of a row where they may not.
  template <typename X>
  __device__ __forceinline__ Raw<X> single(const Tensor& s, const X* src, int c) const {
    Raw<X> v;
    if (s.vec && reinterpret_cast<const uint8_t*>(src + 8) <= s.end) v.load(src);
    else v.gather(src, columns(c));
    return v;
  }
  // Out of line for the rows that need it, which are few.
  template <typename X>
  static __device__ __noinline__ Raw<X> single_call(const uint8_t* end, const X* src, uint32_t on, bool vec) {
    Raw<X> v;
    if (vec && reinterpret_cast<const uint8_t*>(src + 8) <= end) v.load(src);
    else v.gather(src, on);
    return v;
  }
  // The thread's pieces of a row; anything past its ends.  Where vectors may not
  // be read, anything at all, for `mend` to put right when the row is used: a
  // branch around the loads would keep the compiler from moving other work past them.
  template <typename X>
  __device__ __forceinline__ void load(const Tensor& s, long long row, Raw<X> (&q)[P]) const {
    const X* at = static_cast<const X*>(s.base) + row * s.ld + 8 * t - off;
    const bool ok = vectors<X>(s, row);
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (piece(i) < pieces) q[i].load(ok ? at + 8 * i * nt : reinterpret_cast<const X*>(g_zeros));
  }
  template <typename X>
  __device__ __forceinline__ void mend(const Tensor& s, long long row, Raw<X> (&q)[P]) const {
    if (!ODD || vectors<X>(s, row)) return;
    const X* at = static_cast<const X*>(s.base) + row * s.ld + 8 * t - off;
#pragma unroll
    for (int i = 0; i < P; ++i)
      if (piece(i) < pieces) q[i] = single_call<X>(s.end, at + 8 * i * nt, columns(piece(i)), s.vec);
  }
  // Piece c of a row of an output.
  template <typename X>
  __device__ __forceinline__ void store(const Tensor& o, long long row, int c, const Pair (&q)[4]) const {
    X* at = static_cast<X*>(o.base) + row * o.ld + 8 * c - off;
    Raw<X> v;
    v.set(q);
    if (!ODD || (o.vec && whole(c))) v.store(at);
    else v.store(at, max(0, off - 8 * c), min(8, p.D + off - 8 * c), o.vec);
  }
  // ... of one in BF16, zeros where `m` has them.
  __device__ __forceinline__ void store(const Tensor& o, long long row, int c, const Pair (&q)[4], const uint4& m) const {
    __nv_bfloat16* at = static_cast<__nv_bfloat16*>(o.base) + row * o.ld + 8 * c - off;
    Raw<__nv_bfloat16> v;
    v.set(q);
    v.keep(m);
    if (!ODD || (o.vec && whole(c))) v.store(at);
    else v.store(at, max(0, off - 8 * c), min(8, p.D + off - 8 * c), o.vec);
  }
  // Which of the row's elements dropout keeps: keep_words of each piece.
  __device__ __forceinline__ void draw(const PhiloxKey<false>& key, long long row, uint4 (&m)[P]) const {
    const unsigned long long group0 = static_cast<unsigned long long>(row * p.D) >> 3;
#pragma unroll
    for (int i = 0; i < P; ++i) m[i] = keep_words(p.drop, philox(key, group0 + piece(i)));
  }
};

// Thread t of n draws its share of a row's mask: the generator's blocks as they
// are, which the row's own threads compare with the threshold.
__device__ __forceinline__ void draw_row(const LnParams& p, const PhiloxKey<true>& key, long long row, int pieces, int t,
                                         int n, uint4* masks) {
  const unsigned long long group0 = static_cast<unsigned long long>(row * p.D) >> 3;
#pragma unroll 7
  for (int c = t; c < pieces; c += n) masks[c] = philox(key, group0 + c);
}

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
// Fill it (all threads; ends with a barrier).  Plain loads: what ran before may have written the parameters while this
// kernel was in place already, so they are not constant for as long as it is there.
template <int N>
__device__ __forceinline__ void make_table(const LnParams& p, uint8_t* shared, int off, int pieces, int planes) {
  for (int c = threadIdx.x; c < pieces; c += blockDim.x) {
#pragma unroll
    for (int which = 0; which < N; ++which) {
      const void* src = which ? p.bias : p.weight;
      float v[8];
      if (src && off == 0 && 8 * c + 8 <= p.D) {
        if (p.params_f32) {
          const float4 a = static_cast<const float4*>(src)[2 * c];
          const float4 b = static_cast<const float4*>(src)[2 * c + 1];
          v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
        } else {
          const uint4 u = static_cast<const uint4*>(src)[c];
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

// ALL: a branch is there and y is written (the common call): a test around a
// row's loads or stores keeps the compiler from moving anything past it, which
// costs 17 % (8192 x 7168 without dropout: 72.9 and 84.1 us).
// APART: one group, and other warps draw the masks.  That of its k-th row is in
// buffer k mod 2 when the group meets at the second sum of the row before; the
// buffer is written again after the meeting of row k itself, by which it was read.
template <typename R, int P, bool ODD, bool DROP, bool ALL, bool APART = false>
__global__ void __launch_bounds__(fwd_threads(ODD || APART, DROP), 1)
    layer_norm_fwd_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) float red_all[kMaxGroups][128];
  Group<P, ODD> g(p, red_all);
  wait_previous();
  const int planes = (p.D + 7 + (ODD ? 7 : 0)) >> 3;
  const long long step = static_cast<long long>(gridDim.x) * p.groups;
  uint4* const first_mask = reinterpret_cast<uint4*>(shared + p.masks);
  if (APART && g.grp > 0) {
    const PhiloxKey<true> key = philox_key<true>(p.drop);
    const int t = threadIdx.x - 32 * p.warps, n = 32 * p.drawers;
    long long row = blockIdx.x;
    draw_row(p, key, row, g.pieces, t, n, first_mask);
    make_table<2>(p, shared, g.off, g.pieces, planes);
    for (int k = 1; row < p.T; ++k) {
      row += step;
      if (row < p.T) draw_row(p, key, row, g.pieces, t, n, first_mask + (k & 1) * planes);
      named_bar_sync(kSecondBarrier, g.nt + n);
    }
    return;
  }
  const uint4* masks = first_mask;
  long long row = g.grp * gridDim.x + blockIdx.x;
  const bool has_o = ALL || p.o.base != nullptr;
  Raw<R> x[P];
  Raw<__nv_bfloat16> o[P];
  uint4 keep[P];
  if (row < p.T) {
    g.load(p.x, row, x);
    if (has_o) g.load(p.o, row, o);
  }
  PhiloxKey<false> key{};
  if (DROP && !APART) {
    key = philox_key<false>(p.drop);
    g.draw(key, row, keep);
  }
  make_table<2>(p, shared, g.off, g.pieces, planes);
  const float inv_d = 1.0f / static_cast<float>(p.D), beta = p.beta * p.drop.scale;
  for (; row < p.T; row += step) {
    g.mend(p.x, row, x);
    if (has_o) g.mend(p.o, row, o);
    Pair y[P][4], s = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (g.piece(i) >= g.pieces) continue;
      x[i].get(y[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i][j] = mul2(y[i][j], both(p.alpha));
      if (has_o) {
        Pair b[4];
        if (APART) keep[i] = keep_words(p.drop, masks[g.piece(i)]);
        if (DROP) o[i].keep(keep[i]);
        o[i].get(b);
#pragma unroll
        for (int j = 0; j < 4; ++j) y[i][j] = fma2(b[j], both(beta), y[i][j]);
      }
      g.mask(g.piece(i), y[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s = add2(s, y[i][j]);
    }
    if (row + step < p.T) {
      g.load(p.x, row + step, x);
      if (has_o) g.load(p.o, row + step, o);
    }
    if (ALL || p.out0.base) {
#pragma unroll
      for (int i = 0; i < P; ++i)
        if (g.piece(i) < g.pieces) g.template store<R>(p.out0, row, g.piece(i), y[i]);
    }
    const float mean = g.sum(sum2(s)) * inv_d;
    s = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      if (g.piece(i) >= g.pieces) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) y[i][j] = add2(y[i][j], both(-mean));
      g.mask(g.piece(i), y[i]);
#pragma unroll
      for (int j = 0; j < 4; ++j) s = fma2(y[i][j], y[i][j], s);
    }
    const float var = APART ? g.sum(sum2(s), kSecondBarrier + g.grp, g.nt + 32 * p.drawers) : g.sum(sum2(s));
    const float r = inv_sqrt(fmaf(var, inv_d, p.eps));
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
    if (APART) masks = first_mask + (masks == first_mask ? planes : 0);
    if (DROP && !APART) g.draw(key, row + step, keep);   // while the next row is on its way
  }
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void cp_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// A group's rows in flight: y, dh and dy in a ring of slots in shared memory.  A
// thread copies just the pieces it will read itself, so nothing but its own
// copies has to be waited for.
template <typename R, int P, bool ODD, bool ALL>
struct Ring {
  const LnParams& p;
  const Group<P, ODD>& g;
  uint8_t* slots;
  int planes, fill, take;
  long long next;         // row to send for
  long long step;

  __device__ __forceinline__ Ring(const LnParams& p_, const Group<P, ODD>& g_, uint8_t* base, int planes_, long long first,
                                  long long step_)
      : p(p_), g(g_), slots(base + static_cast<size_t>(g_.grp) * p_.stages * p_.slot), planes(planes_), fill(0), take(-1),
        next(first), step(step_) {
    for (int i = 0; i < p.stages; ++i) send();
  }
  template <typename X>
  __device__ __forceinline__ void copy(const Tensor& s, uint8_t* to) const {
    const X* at = static_cast<const X*>(s.base) + next * s.ld + 8 * g.t - g.off;
    X* dst = reinterpret_cast<X*>(to) + 8 * g.t;
    const bool vectors = g.template vectors<X>(s, next);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
      const X* src = at + 8 * i * g.nt;
      if (vectors) {
        const uint32_t d = smem_u32(dst + 8 * i * g.nt);
        cp_async16(d, src);
        if (sizeof(X) == 4) cp_async16(d + 16, src + 4);
      } else {
        *reinterpret_cast<Raw<X>*>(dst + 8 * i * g.nt) = g.template single<X>(s, src, c);
      }
    }
  }
  __device__ __forceinline__ void send() {
    if (next < p.T) {
      uint8_t* to = slots + fill * p.slot;
      copy<R>(p.x, to);
      copy<__nv_bfloat16>(p.dh, to + planes * 8 * sizeof(R));
      if (ALL || p.dy.base) copy<R>(p.dy, to + planes * 8 * (sizeof(R) + 2));
      next += step;
      fill = fill + 1 == p.stages ? 0 : fill + 1;
    }
    cp_commit();
  }
  // Make the next row ready: its slot.
  __device__ __forceinline__ const uint8_t* wait() {
    take = take + 1 == p.stages ? 0 : take + 1;
    if (p.stages == 1) cp_wait<0>();
    else if (p.stages == 2) cp_wait<1>();
    else if (p.stages == 3) cp_wait<2>();
    else cp_wait<3>();
    return slots + take * p.slot;
  }
};

// ALL: dy is there, dx and dbranch are wanted (the common call).
// APART: one group, and the warps that it leaves draw the masks.  The mask of its
// k-th row is in buffer k mod 2 when the group meets at that row's sums; the
// buffer is written again after the next row's meeting, by which it was read.
template <typename R, int P, bool ODD, bool DROP, bool ALL, bool APART = false>
__global__ void __launch_bounds__(kBwdThreads, 1) layer_norm_bwd_kernel(const __grid_constant__ LnParams p) {
  extern __shared__ __align__(16) uint8_t shared[];
  __shared__ __align__(16) float red_all[kMaxGroups][128];
  Group<P, ODD> g(p, red_all);
  wait_previous();
  const int planes = (p.D + 7 + (ODD ? 7 : 0)) >> 3;
  const long long step = static_cast<long long>(gridDim.x) * p.groups;
  long long row = g.grp * gridDim.x + blockIdx.x;
  uint4* const first_mask = reinterpret_cast<uint4*>(shared + p.masks);
  uint4* masks = first_mask;
  const bool drawer = APART && g.grp > 0;
  if (APART) g.members += 32 * p.drawers;
  Ring<R, P, ODD, ALL> ring(p, g, shared + planes * 32, planes, drawer ? p.T : row, step);
  float mean = 0.0f, r = 0.0f;
  if (row < p.T) {
    mean = p.stats[row];
    r = p.stats[p.T + row];
  }
  PhiloxKey<false> key{};
  uint4 keep[P];
  if (DROP && !APART) {
    key = philox_key<false>(p.drop);
    g.draw(key, row, keep);
  }
  if (drawer) {
    const PhiloxKey<true> all = philox_key<true>(p.drop);
    const int t = threadIdx.x - 32 * p.warps, n = 32 * p.drawers;
    row = blockIdx.x;
    draw_row(p, all, row, g.pieces, t, n, masks);
    make_table<1>(p, shared, g.off, g.pieces, planes);
    for (int k = 1; row < p.T; ++k) {
      named_bar_sync(1, g.members);
      row += step;
      if (row < p.T) draw_row(p, all, row, g.pieces, t, n, masks + (k & 1) * planes);
    }
  } else {
    make_table<1>(p, shared, g.off, g.pieces, planes);
  }
  const float inv_d = 1.0f / static_cast<float>(p.D), beta = p.beta * p.drop.scale;
  Pair sw[P][4], sb[P][4];   // sums over the group's rows of dh n and dh
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < 4; ++j) sw[i][j] = sb[i][j] = both(0.0f);
  for (; row < p.T; row += step) {
    const uint8_t* slot = ring.wait();
    const Pair r2 = both(r), mr = both(-mean * r);
    if (row + step < p.T) {   // the next row's
      mean = p.stats[row + step];
      r = p.stats[p.T + row + step];
    }
    Pair n[P][4], a[P][4], sa = both(0.0f), san = both(0.0f);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
      Raw<R> y;
      Raw<__nv_bfloat16> dh;
      y.load(reinterpret_cast<const R*>(slot) + 8 * c);
      dh.load(reinterpret_cast<const __nv_bfloat16*>(slot + planes * 8 * sizeof(R)) + 8 * c);
      if (ODD && !g.whole(c)) {
        y.only(g.columns(c));
        dh.only(g.columns(c));
      }
      Pair w[4];
      y.get(n[i]);
      dh.get(a[i]);
      table_load(shared, planes, 0, c, w);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        n[i][j] = fma2(n[i][j], r2, mr);
        sb[i][j] = add2(sb[i][j], a[i][j]);
        sw[i][j] = fma2(a[i][j], n[i][j], sw[i][j]);
        a[i][j] = mul2(a[i][j], w[j]);
        sa = add2(sa, a[i][j]);
        san = fma2(a[i][j], n[i][j], san);
      }
    }
    float ma = sum2(sa), man = sum2(san);
    g.sum_two(ma, man);
    float rr, unused;
    split(r2, rr, unused);
    const Pair rma = both(-rr * ma * inv_d), rman = both(-rr * man * inv_d);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = g.piece(i);
      if (c >= g.pieces) continue;
      Pair s[4];
      if (ALL || p.dy.base) {
        Raw<R> dy;
        dy.load(reinterpret_cast<const R*>(slot + planes * 8 * (sizeof(R) + 2)) + 8 * c);
        dy.get(s);
      } else {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = both(0.0f);
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        s[j] = fma2(n[i][j], rman, fma2(a[i][j], r2, add2(s[j], rma)));
        n[i][j] = mul2(s[j], both(p.alpha));
      }
      if (ALL || p.out0.base) g.template store<R>(p.out0, row, c, n[i]);
      if (ALL || p.out1.base) {
#pragma unroll
        for (int j = 0; j < 4; ++j) s[j] = mul2(s[j], both(beta));
        if (APART) keep[i] = keep_words(p.drop, masks[c]);
        if (DROP) g.store(p.out1, row, c, s, keep[i]);
        else g.template store<__nv_bfloat16>(p.out1, row, c, s);
      }
    }
    ring.send();
    if (APART) masks = first_mask + (masks == first_mask ? planes : 0);
    if (DROP && !APART) g.draw(key, row + step, keep);   // while the next row is on its way
  }
  cp_wait<0>();
  __syncthreads();   // the rows' memory is free: it takes the groups' sums
  float4* acc = reinterpret_cast<float4*>(shared) + 2 * planes;   // [2 arrays][2 halves][planes], when groups > 1
  for (int k = 0; k < p.groups; ++k) {
    if (k == g.grp) {
#pragma unroll
      for (int arr = 0; arr < 2; ++arr) {
        // in the layout's pieces, shifted like the rows
        float4* out = reinterpret_cast<float4*>(p.partial) +
                      (static_cast<long long>(arr) * gridDim.x + blockIdx.x) * 2 * planes;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const int c = g.piece(i);
          if (c >= g.pieces) continue;
          Pair b[4];
          if (k > 0) table_load(reinterpret_cast<uint8_t*>(acc), planes, arr, c, b);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const Pair v = arr == 0 ? sw[i][j] : sb[i][j];
            b[j] = k > 0 ? add2(b[j], v) : v;
          }
          float v[8];
#pragma unroll
          for (int j = 0; j < 4; ++j) split(b[j], v[2 * j], v[2 * j + 1]);
          const bool last = k + 1 == p.groups;
          float4* lo = last ? out + 2 * c : table_at(reinterpret_cast<uint8_t*>(acc), planes, arr, 0, c);
          float4* hi = last ? lo + 1 : lo + planes;
          *lo = make_float4(v[0], v[1], v[2], v[3]);
          *hi = make_float4(v[4], v[5], v[6], v[7]);
        }
      }
    }
    if (k + 1 < p.groups) __syncthreads();
  }
}

// The CTAs' column sums joined in a fixed order (eight interleaved sums a
// column, then those in order): blockIdx.y = 0 dweight, 1 dbias.
__global__ void __launch_bounds__(256) layer_norm_sums_kernel(const float* partial, int rows, int D, int pitch,
                                                              float* dweight, float* dbias) {
  __shared__ float part[8][33];
  wait_previous();
  float* out = blockIdx.y ? dbias : dweight;
  if (out == nullptr) return;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.0f;
  if (c < D) {
    const float* q = partial + static_cast<long long>(blockIdx.y) * rows * pitch + c;
    // CTA r's columns are shifted like its rows
#pragma unroll 8
    for (int r = ry; r < rows; r += 8) s += q[static_cast<long long>(r) * pitch + (r * (D & 7) & 7)];
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
Tensor tensor(const LnParams& p, const void* base, int64_t ld, int esz) {
  const long long l = ld ? ld : p.D;
  return {const_cast<void*>(base), l, (l - p.D) % 8 == 0 || p.T == 1,
          static_cast<const uint8_t*>(base) + ((p.T - 1) * l + p.D) * esz};
}

constexpr int kSmem = 216 * 1024;   // the columns' factors and the backward's rows in flight

struct Shape {
  int pieces, ctas, threads;
  int row_pieces;      // pieces of a row, at most
  bool odd;
  bool apart;          // the masks are drawn by warps of their own
  size_t smem;
};

// Pieces a thread, warps a row, groups a CTA.
Shape place(LnParams* p, bool fwd, int esz, int sms) {
  Shape s;
  const bool ragged = p->D % 8 != 0;
  s.odd = ragged;
  for (const Tensor* t : {&p->x, &p->o, &p->dy, &p->dh, &p->out0, &p->out1}) s.odd = s.odd || (t->base && !t->vec);
  const int all = s.row_pieces = (p->D + 7 + (s.odd ? 7 : 0)) / 8;
  // One piece a thread where a warp holds the row, and where an FP32 residual's two would not fit the forward's registers
  // beside the other group's (16384 x 2048 without dropout 62.7 and 73.8 us; with it 73.3 and 68.6); four for the odd
  // widths next to the limit, which two do not hold.
  s.pieces = all <= 32 || (fwd && esz == 4 && !p->drop.rng && all <= fwd_threads(s.odd, false)) ? 1 : all <= 1024 ? 2 : 4;
  p->warps = (all + 32 * s.pieces - 1) / (32 * s.pieces);
  int most = std::min((fwd ? fwd_threads(s.odd, p->drop.rng != nullptr) : kBwdThreads) / 32 / p->warps, kMaxGroups);
  const int room = kSmem - all * 32;
  if (!fwd) {
    p->slot = all * 8 * (2 * esz + 2);
    most = std::max(1, std::min(most, room / (2 * p->slot)));   // two rows in flight a group at least, where they fit
  }
  // no more groups than save a round of rows
  const int rounds = (p->T - 1) / (sms * most) + 1;
  p->groups = (p->T - 1) / (sms * rounds) + 1;
  // Dropout where a row takes so many of 16 warps that the CTA has one group, but leaves two: these draw the masks.
  // Backward 2048 x 7168, two warps: 43.3 and 36.5 us, 150 rows 10.4 and 9.9; 4096 x 4352, seven: 56 and 46; one warp is
  // not enough: 4096 x 7680 75 and 89.  Forward, which has two groups otherwise: 2048 x 7168 27.4 and 26.3 us, 300 rows 8.0
  // and 6.3, 8192 90.4 and 91.8, 4096 x 6144 both 42.6, 4096 x 5120 37.6 and 38.7; FP32 4096 x 7168 67.0 and 60.9, 4096 x
  // 5120 50.3 and 48.5, 4096 x 4352 41.2 and 42.6.
  const int spare = 16 - p->warps;
  s.apart = p->drop.rng && !s.odd && s.pieces == 2 && spare >= 2 && p->out0.base &&
            (fwd ? p->o.base && p->warps > (esz == 4 ? 9 : 12)
                 : p->warps > 1 && p->groups == 1 && p->dy.base && p->out1.base);
  if (s.apart) p->groups = 1;
  p->drawers = s.apart ? spare : 0;
  s.threads = (p->warps * p->groups + p->drawers) * 32;
  // a group's rows have to be a multiple of 8 apart
  s.ctas = !ragged || p->T <= sms ? std::min(sms, p->T) : std::max(8, sms / 8 * 8);
  // the columns' factors; backward: the rows in flight, whose place the groups' sums take
  const int masks = s.apart ? 2 * all * 16 : 0;
  p->masks = 2 * all * 32;
  s.smem = p->masks + masks;
  if (!fwd) {
    p->stages = std::max(1, std::min(4, (room - masks) / (p->groups * p->slot)));
    p->masks = all * 32 + std::max(p->groups > 1 ? all * 64 : 0, p->groups * p->stages * p->slot);
    s.smem = p->masks + masks;
  }
  return s;
}

template <typename K>
cudaError_t launch(K kernel, PerDeviceOnce& once, const Shape& s, const LnParams& p, cudaStream_t stream) {
  const cudaError_t e =
      once.once([&] { return cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem); });
  if (e != cudaSuccess) return e;
  void* args[] = {const_cast<LnParams*>(&p)};
  return launch_dependent(reinterpret_cast<const void*>(kernel), dim3(s.ctas), s.threads, s.smem, stream, args);
}

template <typename R, int P, bool ODD, bool DROP>
cudaError_t launch_as(bool fwd, const Shape& s, const LnParams& p, cudaStream_t stream) {
  static PerDeviceOnce f, b, f_all, b_all;
  if constexpr (P == 2 && !ODD && DROP) {
    static PerDeviceOnce f_apart, b_apart;
    if (s.apart)
      return fwd ? launch(layer_norm_fwd_kernel<R, P, ODD, DROP, true, true>, f_apart, s, p, stream)
                 : launch(layer_norm_bwd_kernel<R, P, ODD, DROP, true, true>, b_apart, s, p, stream);
  }
  if (fwd)
    return p.o.base && p.out0.base ? launch(layer_norm_fwd_kernel<R, P, ODD, DROP, true>, f_all, s, p, stream)
                                   : launch(layer_norm_fwd_kernel<R, P, ODD, DROP, false>, f, s, p, stream);
  return p.dy.base && p.out0.base && p.out1.base ? launch(layer_norm_bwd_kernel<R, P, ODD, DROP, true>, b_all, s, p, stream)
                                                 : launch(layer_norm_bwd_kernel<R, P, ODD, DROP, false>, b, s, p, stream);
}
template <typename R, int P>
cudaError_t launch_p(bool fwd, const Shape& s, const LnParams& p, cudaStream_t stream) {
  const bool drop = p.drop.rng != nullptr;
  if (s.odd) return drop ? launch_as<R, P, true, true>(fwd, s, p, stream) : launch_as<R, P, true, false>(fwd, s, p, stream);
  return drop ? launch_as<R, P, false, true>(fwd, s, p, stream) : launch_as<R, P, false, false>(fwd, s, p, stream);
}
template <typename R>
cudaError_t launch_r(bool fwd, const Shape& s, const LnParams& p, cudaStream_t stream) {
  if (s.pieces == 1) return launch_p<R, 1>(fwd, s, p, stream);
  if (s.pieces == 2) return launch_p<R, 2>(fwd, s, p, stream);
  return p.drop.rng ? launch_as<R, 4, true, true>(fwd, s, p, stream) : launch_as<R, 4, true, false>(fwd, s, p, stream);
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
  const int esz = f32 ? 4 : 2;
  p.weight = weight;
  p.bias = bias;
  p.stats = stats;
  p.x = tensor(p, x, cfg->x_stride, esz);
  p.o = tensor(p, branch, cfg->branch_stride, 2);
  p.out0 = tensor(p, y, cfg->y_stride, esz);
  p.out1 = tensor(p, h, cfg->h_stride, 2);
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const Shape s = place(&p, true, esz, sms);
  return launch_norm(true, f32, s, p, stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_layer_norm_workspace_bytes(const moe_layer_norm_config* cfg) {
  if (!config_ok(cfg) || cfg->d_model > kMaxCols) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  // two arrays of column sums a CTA
  const size_t rows = static_cast<size_t>(std::min(cfg->tokens, std::max(8, sms)));
  return 2 * rows * static_cast<size_t>((cfg->d_model + 14) / 8 * 8) * sizeof(float) + 256;
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
  const int esz = f32 ? 4 : 2;
  p.weight = weight;
  p.stats = const_cast<float*>(stats);
  p.partial = static_cast<float*>(workspace);
  p.x = tensor(p, y, cfg->x_stride, esz);
  p.dh = tensor(p, dh, cfg->h_stride, 2);
  p.dy = tensor(p, dy, cfg->y_stride, esz);
  p.out0 = tensor(p, dx, 0, esz);
  p.out1 = tensor(p, dbranch, 0, 2);
  const Shape s = place(&p, false, esz, sms);
  if (launch_norm(false, f32, s, p, stream) != cudaSuccess) return MOE_ERR_CUDA;
  if (dweight || dbias) {
    const float* partial = p.partial;
    int rows = s.ctas, d = D, pitch = 8 * s.row_pieces;
    void* args[] = {&partial, &rows, &d, &pitch, &dweight, &dbias};
    if (launch_dependent(reinterpret_cast<const void*>(layer_norm_sums_kernel), dim3((D + 31) / 32, 2), 256, 0, stream,
                         args) != cudaSuccess)
      return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
