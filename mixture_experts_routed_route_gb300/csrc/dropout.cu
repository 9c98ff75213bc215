// Dropout from a counter-based generator (moe_dropout): out = keep x / (1 - p)
// (+ residual), and, called with the gradient in x's place and the same rng
// and site, its own backward.  The mask is that of philox.cuh, by element of
// the [T, D] tensor, whatever its strides.
//
// A thread takes groups of eight elements, which share one block of the
// generator, kBatch of them with all loads sent first.  What bounds it is the
// stream, once long.
#include <algorithm>

#include "kernels.cuh"
#include "moe_gb300.h"
#include "philox.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kBatch = 4;

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

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
  const uint4 u = *reinterpret_cast<const uint4*>(p);
  v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
  v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
  const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
  v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[8]) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                            pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[8]) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}
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

template <typename X, int LAYOUT>
__global__ void __launch_bounds__(kThreads) dropout_kernel(const __grid_constant__ DropoutParams p) {
  const X* x = static_cast<const X*>(p.x);
  const X* res = static_cast<const X*>(p.residual);
  X* out = static_cast<X*>(p.out);
  const bool drop = p.drop.rng != nullptr;
  PhiloxKey key{};
  if (drop) key = philox_key(p.drop);
  const long long g0 = static_cast<long long>(blockIdx.x) * (kThreads * kBatch) + threadIdx.x;
  if constexpr (LAYOUT == kAny) {
    for (int b = 0; b < kBatch; ++b) {
      const long long g = g0 + b * kThreads;
      if (g >= p.groups) return;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (drop) w = philox(key, g);
      long long t = g * 8 / p.D;
      int d = static_cast<int>(g * 8 - t * p.D);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        if (g * 8 + j >= p.n) return;
        float v = to_f(x[t * p.ldx + d]);
        v = !drop || kept(w, j, p.drop.threshold) ? v * p.drop.scale : 0.0f;
        if (res) v += to_f(res[t * p.ldr + d]);
        put(out + t * p.ldo + d, v);
        if (++d == p.D) {
          d = 0;
          ++t;
        }
      }
    }
    return;
  } else {
    long long at[kBatch][3];
    bool on[kBatch];
    float v[kBatch][8], r[kBatch][8];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const long long g = g0 + b * kThreads;
      on[b] = (g + 1) * 8 <= p.n;
      if constexpr (LAYOUT == kFlat) {
        at[b][0] = at[b][1] = at[b][2] = g * 8;
      } else {
        const long long t = g / p.row_groups;
        const long long d = (g - t * p.row_groups) * 8;
        at[b][0] = t * p.ldx + d;
        at[b][1] = t * p.ldr + d;
        at[b][2] = t * p.ldo + d;
      }
      if (on[b]) load8(x + at[b][0], v[b]);
    }
    if (res) {
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
        if (on[b]) load8(res + at[b][1], r[b]);
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const long long g = g0 + b * kThreads;
      if (g >= p.groups) continue;
      uint4 w = make_uint4(0, 0, 0, 0);
      if (drop) w = philox(key, g);
      if (on[b]) {
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          v[b][j] = !drop || kept(w, j, p.drop.threshold) ? v[b][j] * p.drop.scale : 0.0f;
          if (res) v[b][j] += r[b][j];
        }
        store8(out + at[b][2], v[b]);
      } else {   // the last elements of a flat tensor
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const long long e = g * 8 + j;
          if (e < p.n) {
            float u = !drop || kept(w, j, p.drop.threshold) ? to_f(x[e]) * p.drop.scale : 0.0f;
            if (res) u += to_f(res[e]);
            put(out + e, u);
          }
        }
      }
    }
  }
}

template <typename X>
void launch(int layout, unsigned grid, const DropoutParams& p, cudaStream_t stream) {
  if (layout == kFlat) dropout_kernel<X, kFlat><<<grid, kThreads, 0, stream>>>(p);
  else if (layout == kRows) dropout_kernel<X, kRows><<<grid, kThreads, 0, stream>>>(p);
  else dropout_kernel<X, kAny><<<grid, kThreads, 0, stream>>>(p);
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
  const long long per = kThreads * kBatch, grid = (p.groups + per - 1) / per;
  if (grid > 0x7FFFFFFFll) return MOE_ERR_UNSUPPORTED;
  if (cfg->type == MOE_TYPE_FP32) launch<float>(layout, static_cast<unsigned>(grid), p, stream);
  else launch<__nv_bfloat16>(layout, static_cast<unsigned>(grid), p, stream);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // extern "C"
