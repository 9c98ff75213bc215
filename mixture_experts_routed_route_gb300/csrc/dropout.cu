// Dropout from a counter-based generator (moe_dropout): out = keep x / (1 - p)
// (+ residual), and, called with the gradient in x's place and the same rng
// and site, its own backward.  The mask is that of philox.cuh, by element of
// the [T, D] tensor, whatever its strides.
//
// A thread takes groups of eight elements, which share one block of the
// generator, one after the other, the next one's loads ahead of this one's mask.
// What bounds it: the stream (16384 x 7168 in BF16 77 us, 6.1 TB/s, floor 69; FP32
// 135 us, 6.9 TB/s).  Beside it the generator's 32 x 32 -> 64 bit products, 19 a
// group at 4 cycles a warp and scheduler, take 29 us, and 60 % of the issue slots
// are busy in BF16.  On the way there, BF16:
// four groups a thread at a time with 98 registers took 133 us (22 % of the warps:
// products and logic, which run in different pipes, hardly overlapped); the first
// round's product with the site is formed once a thread, and dropped places are
// cleared in the packed words.
#include <algorithm>

#include "kernels.cuh"
#include "moe_gb300.h"
#include "philox.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
// CTAs an SM at most, of which six or so run at a time: a few groups a thread
// spread the keys' cost, and many CTAs keep the SMs evenly busy (16384 x 7168 in
// BF16: 8 an SM 79.9 us, 16 78.4, 64 77.6; in FP32 148, 147, 139).
constexpr int kCtas = 64;

struct DropoutParams {
  long long groups;          // of eight elements
  long long n;               // elements, T D
  int D;
  int row_groups;            // rows of vectors: D / 8
  long long ldx, ldr, ldo;
  const void* x;
  const void* residual;      // or NULL
  void* out;
  DropParams drop;
};

// Eight elements as they lie in memory.
template <typename X>
struct Raw;
template <>
struct Raw<__nv_bfloat16> {
  uint4 u;
  __device__ __forceinline__ void load(const __nv_bfloat16* p) { u = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void store(__nv_bfloat16* p) const { *reinterpret_cast<uint4*>(p) = u; }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    u = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
  }
  // zeros where dropped, on the packed words: after the rounding, two elements an instruction
  __device__ __forceinline__ void drop(const uint4& m) { u = make_uint4(u.x & m.x, u.y & m.y, u.z & m.z, u.w & m.w); }
};
template <>
struct Raw<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float* p) {
    a = reinterpret_cast<const float4*>(p)[0];
    b = reinterpret_cast<const float4*>(p)[1];
  }
  __device__ __forceinline__ void store(float* p) const {
    reinterpret_cast<float4*>(p)[0] = a;
    reinterpret_cast<float4*>(p)[1] = b;
  }
  __device__ __forceinline__ void get(float (&v)[8]) const {
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  }
  __device__ __forceinline__ void set(const float (&v)[8]) {
    a = make_float4(v[0], v[1], v[2], v[3]);
    b = make_float4(v[4], v[5], v[6], v[7]);
  }
  __device__ __forceinline__ void drop(const uint4& m) {
    float v[8];
    get(v);
#pragma unroll
    for (int j = 0; j < 8; ++j)
      if (!kept(m, j)) v[j] = 0.0f;
    set(v);
  }
};
__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// How a group of eight elements lies in memory.
enum Layout {
  kFlat,    // all tensors contiguous: one vector, but for the last n % 8 elements
  kRows,    // D and the strides multiples of 8: one vector of a row
  kAny      // element by element
};

// Group g element by element.
template <typename X>
__device__ __forceinline__ void scalar_group(const DropoutParams& p, const PhiloxKey<true>& key, long long g) {
  uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
  if (p.drop.rng) m = keep_words(p.drop, philox(key, g));
  long long t = g * 8 / p.D;
  int d = static_cast<int>(g * 8 - t * p.D);
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    if (g * 8 + j >= p.n) return;
    float v = to_f(static_cast<const X*>(p.x)[t * p.ldx + d]);
    v = kept(m, j) ? v * p.drop.scale : 0.0f;
    if (p.residual) v += to_f(static_cast<const X*>(p.residual)[t * p.ldr + d]);
    put(static_cast<X*>(p.out) + t * p.ldo + d, v);
    if (++d == p.D) {
      d = 0;
      ++t;
    }
  }
}

template <typename X, int LAYOUT, bool RES>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutParams p) {
  const X* x = static_cast<const X*>(p.x);
  const X* res = static_cast<const X*>(p.residual);
  X* out = static_cast<X*>(p.out);
  const long long hop = static_cast<long long>(gridDim.x) * kThreads;
  long long g = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
  wait_previous();
  PhiloxKey<true> key{};
  if (p.drop.rng) key = philox_key<true>(p.drop);
  if constexpr (LAYOUT == kAny) {
    for (; g < p.groups; g += hop) scalar_group<X>(p, key, g);
  } else {
    // row and group in the row, moved on by adding: no division in the loop
    long long t = 0, d = g, hop_t = 0, hop_d = hop;
    if (LAYOUT == kRows) {
      t = g / p.row_groups;
      d = g - t * p.row_groups;
      hop_t = hop / p.row_groups;
      hop_d = hop - hop_t * p.row_groups;
    }
    const long long whole = p.n / 8;
    Raw<X> v, r;
    if (g < whole) {
      v.load(x + t * p.ldx + d * 8);
      if (RES) r.load(res + t * p.ldr + d * 8);
    }
    for (; g < whole; g += hop) {
      X* o = out + t * p.ldo + d * 8;
      t += hop_t;
      d += hop_d;
      if (LAYOUT == kRows && d >= p.row_groups) {
        d -= p.row_groups;
        ++t;
      }
      Raw<X> nv, nr;   // the next group is on its way while this one's mask is drawn
      if (g + hop < whole) {
        nv.load(x + t * p.ldx + d * 8);
        if (RES) nr.load(res + t * p.ldr + d * 8);
      }
      uint4 m = make_uint4(~0u, ~0u, ~0u, ~0u);
      if (p.drop.rng) m = keep_words(p.drop, philox(key, g));
      float f[8];
      v.get(f);
      if constexpr (RES) {
        float s[8];
        r.get(s);
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] = kept(m, j) ? fmaf(f[j], p.drop.scale, s[j]) : s[j];
        v.set(f);
      } else {
#pragma unroll
        for (int j = 0; j < 8; ++j) f[j] *= p.drop.scale;
        v.set(f);
        v.drop(m);
      }
      v.store(o);
      v = nv;
      r = nr;
    }
    if (LAYOUT == kFlat && g == whole && g < p.groups) scalar_group<X>(p, key, g);   // the last elements
  }
}

template <typename X>
const void* kernel_of(int layout, bool residual) {
  if (layout == kAny) return reinterpret_cast<const void*>(dropout_kernel<X, kAny, false>);
  if (layout == kFlat)
    return residual ? reinterpret_cast<const void*>(dropout_kernel<X, kFlat, true>)
                    : reinterpret_cast<const void*>(dropout_kernel<X, kFlat, false>);
  return residual ? reinterpret_cast<const void*>(dropout_kernel<X, kRows, true>)
                  : reinterpret_cast<const void*>(dropout_kernel<X, kRows, false>);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_dropout(const moe_dropout_config* cfg, const void* x, const void* residual, const int64_t* rng, void* out,
                       cudaStream_t stream) {
  if (!cfg || cfg->tokens < 0 || cfg->d_model < 1) return MOE_ERR_INVALID_ARG;
  if (cfg->type != MOE_TYPE_BF16 && cfg->type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  for (int64_t ld : {cfg->x_stride, cfg->residual_stride, cfg->out_stride})
    if (ld != 0 && ld < cfg->d_model) return MOE_ERR_INVALID_ARG;
  DropoutParams p{};
  if (!drop_params(&p.drop, rng, cfg->p, cfg->site)) return MOE_ERR_INVALID_ARG;
  if (cfg->tokens == 0) return MOE_OK;
  if (!x || !out || (p.drop.threshold && !rng)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, residual, static_cast<const void*>(rng), static_cast<const void*>(out)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  p.D = cfg->d_model;
  p.n = static_cast<long long>(cfg->tokens) * p.D;
  p.groups = (p.n + 7) / 8;
  p.row_groups = p.D / 8;
  p.ldx = cfg->x_stride ? cfg->x_stride : p.D;
  p.ldr = cfg->residual_stride ? cfg->residual_stride : p.D;
  p.ldo = cfg->out_stride ? cfg->out_stride : p.D;
  p.x = x;
  p.residual = residual;
  p.out = out;
  if (!residual) p.ldr = p.ldx;
  int layout = kAny;
  if (cfg->tokens == 1 || (p.ldx == p.D && p.ldr == p.D && p.ldo == p.D)) layout = kFlat;
  else if (p.D % 8 == 0 && p.ldx % 8 == 0 && p.ldr % 8 == 0 && p.ldo % 8 == 0) layout = kRows;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const long long grid = std::min<long long>((p.groups + kThreads - 1) / kThreads, kCtas * sms);
  void* args[] = {&p};
  const bool res = residual != nullptr;
  const void* kernel = cfg->type == MOE_TYPE_FP32 ? kernel_of<float>(layout, res) : kernel_of<__nv_bfloat16>(layout, res);
  return launch_dependent(kernel, dim3(static_cast<unsigned>(grid)), kThreads, 0, stream, args) == cudaSuccess ? MOE_OK
                                                                                                              : MOE_ERR_CUDA;
}

}  // extern "C"
