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
// Work layout: a group of W warps owns a row (W = ceil(D / 512), 16 columns
// a thread), so a row stays in registers between its loads and its stores;
// groups of rows narrower than a CTA share one.  A group's row sums go
// through shared memory under a named barrier of its own.
#include "kernels.cuh"
#include "moe_gb300.h"

namespace moe {

namespace {

constexpr int kCols = 16;             // columns per thread
constexpr int kWarpCols = 32 * kCols; // columns per warp
constexpr int kMaxCols = 32 * kWarpCols;

struct NormParams {
  int T, D;
  int warps, groups;          // warps per row, rows in flight per CTA
  const void* x;              // [T, ldx] residual type
  const __nv_bfloat16* o;     // [T, ldo] or NULL
  const void* gate;
  const void* w_post;         // NULL: no norm after the block
  const void* w_pre;          // NULL: no norm before the next
  long long ldx, ldo, ldy, ldh;
  int gate_mode, rows_per_group;
  int params_f32, gate_f32;
  float alpha, beta, eps, offset;
  // forward
  void* y;
  __nv_bfloat16* h;
  float* stats;               // [2][T]: r_o, r_y (backward: read)
  // backward
  const void* dy;             // or NULL
  const __nv_bfloat16* dh;    // or NULL
  void* dx;                   // or NULL
  __nv_bfloat16* do_;
  void* dgate;
  long long lddy, lddh, lddx, lddo;
  float* partial;             // [3][gridDim.x][D]: dw_post, dw_pre, dgate (channel)
  float* gate_partial;        // [slabs][D] (grouped gates cut into several slabs a group)
  int slabs_per_group, slabs;
};

// V consecutive values at p as FP32 (V = 8: one or two 16-byte loads).
template <int V>
__device__ __forceinline__ void load_v(const __nv_bfloat16* p, float* v) {
  if constexpr (V == 8) {
    const uint4 u = *reinterpret_cast<const uint4*>(p);
    v[0] = bf16_lo(u.x), v[1] = bf16_hi(u.x), v[2] = bf16_lo(u.y), v[3] = bf16_hi(u.y);
    v[4] = bf16_lo(u.z), v[5] = bf16_hi(u.z), v[6] = bf16_lo(u.w), v[7] = bf16_hi(u.w);
  } else {
    v[0] = __bfloat162float(*p);
  }
}

template <int V>
__device__ __forceinline__ void load_v(const float* p, float* v) {
  if constexpr (V == 8) {
    const float4 a = reinterpret_cast<const float4*>(p)[0], b = reinterpret_cast<const float4*>(p)[1];
    v[0] = a.x, v[1] = a.y, v[2] = a.z, v[3] = a.w, v[4] = b.x, v[5] = b.y, v[6] = b.z, v[7] = b.w;
  } else {
    v[0] = *p;
  }
}

template <int V>
__device__ __forceinline__ void store_v(__nv_bfloat16* p, const float* v) {
  if constexpr (V == 8)
    *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                                              pack_bf16x2(v[6], v[7]));
  else
    *p = __float2bfloat16_rn(v[0]);
}

template <int V>
__device__ __forceinline__ void store_v(float* p, const float* v) {
  if constexpr (V == 8) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
  } else {
    *p = v[0];
  }
}

// Weights and gates come in either type (a uniform branch).
template <int V>
__device__ __forceinline__ void load_param(const void* p, int f32, long long at, float* v) {
  if (f32) load_v<V>(static_cast<const float*>(p) + at, v);
  else load_v<V>(static_cast<const __nv_bfloat16*>(p) + at, v);
}

template <int V>
__device__ __forceinline__ void store_param(void* p, int f32, long long at, const float* v) {
  if (f32) store_v<V>(static_cast<float*>(p) + at, v);
  else store_v<V>(static_cast<__nv_bfloat16*>(p) + at, v);
}

// Sum over a group's `warps` warps in a fixed order: an xor tree in each
// warp, then the warp sums in warp order.  `red` is the group's 2 x 32
// floats, used in turns (`turn` flips), so one barrier a sum is enough.
__device__ __forceinline__ float group_sum(float v, float* red, int warps, int wig, int bar, int& turn) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if (warps == 1) return v;
  float* r = red + turn * 32;
  turn ^= 1;
  if ((threadIdx.x & 31) == 0) r[wig] = v;
  named_bar_sync(bar, warps * 32);
  float t = 0.0f;
  for (int w = 0; w < warps; ++w) t += r[w];
  return t;
}

__device__ __forceinline__ long long gate_row(const NormParams& p, long long row) {
  return static_cast<long long>(p.gate_mode == MOE_GATE_GROUP ? row / p.rows_per_group : 0) * p.D;
}

// g w_o for V columns from c (1 where there is no gate or no norm).
template <int V>
__device__ __forceinline__ void gate_v(const NormParams& p, long long row, int c, float* g) {
  if (p.gate_mode == MOE_GATE_CHANNEL || p.gate_mode == MOE_GATE_GROUP) {
    load_param<V>(p.gate, p.gate_f32, gate_row(p, row) + c, g);
  } else {
    float t = 1.0f;
    if (p.gate_mode == MOE_GATE_TOKEN) load_param<1>(p.gate, p.gate_f32, row, &t);
#pragma unroll
    for (int j = 0; j < V; ++j) g[j] = t;
  }
}

template <int V>
__device__ __forceinline__ void weight_v(const NormParams& p, const void* w, int c, float* v) {
  if (w == nullptr) {
#pragma unroll
    for (int j = 0; j < V; ++j) v[j] = 1.0f;
    return;
  }
  load_param<V>(w, p.params_f32, c, v);
#pragma unroll
  for (int j = 0; j < V; ++j) v[j] += p.offset;
}

template <typename R, int V, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_fwd_kernel(const NormParams p) {
  constexpr int NV = kCols / V;
  __shared__ float red_all[16][64];
  const int warp = threadIdx.x >> 5;
  const int grp = warp / p.warps, wig = warp - grp * p.warps;
  const int t = threadIdx.x - grp * p.warps * 32, nt = p.warps * 32;
  float* red = red_all[grp];
  int turn = 0;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const long long row = static_cast<long long>(blockIdx.x) * p.groups + grp;
  if (row >= p.T) return;   // a whole group: its barrier has no other members
  const R* x = static_cast<const R*>(p.x) + row * p.ldx;
  float y[kCols], o[kCols];
  float so = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * nt) * V;
#pragma unroll
    for (int j = 0; j < V; ++j) y[i * V + j] = o[i * V + j] = 0.0f;
    if (c < p.D) {
      load_v<V>(x + c, y + i * V);
      if (p.o) load_v<V>(p.o + row * p.ldo + c, o + i * V);
    }
#pragma unroll
    for (int j = 0; j < V; ++j) so = fmaf(o[i * V + j], o[i * V + j], so);
  }
  float r_o = 1.0f;
  if (p.w_post) {
    r_o = 1.0f / sqrtf(group_sum(so, red, p.warps, wig, 1 + grp, turn) * inv_d + p.eps);
    if (p.stats && t == 0) p.stats[row] = r_o;
  }
  float sy = 0.0f;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int c = (t + i * nt) * V;
    if (c < p.D) {
      if (p.o) {
        float w[V], g[V];
        weight_v<V>(p, p.w_post, c, w);
        gate_v<V>(p, row, c, g);
#pragma unroll
        for (int j = 0; j < V; ++j)
          y[i * V + j] = fmaf(p.alpha, y[i * V + j], p.beta * (g[j] * (o[i * V + j] * r_o * w[j])));
      } else {
#pragma unroll
        for (int j = 0; j < V; ++j) y[i * V + j] *= p.alpha;
      }
      if (p.y) store_v<V>(static_cast<R*>(p.y) + row * p.ldy + c, y + i * V);
#pragma unroll
      for (int j = 0; j < V; ++j) sy = fmaf(y[i * V + j], y[i * V + j], sy);
    }
  }
  if (p.w_pre) {
    const float r_y = 1.0f / sqrtf(group_sum(sy, red, p.warps, wig, 1 + grp, turn) * inv_d + p.eps);
    if (p.stats && t == 0) p.stats[p.T + row] = r_y;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * V;
      if (c < p.D) {
        float w[V];
        weight_v<V>(p, p.w_pre, c, w);
#pragma unroll
        for (int j = 0; j < V; ++j) y[i * V + j] = y[i * V + j] * r_y * w[j];
        store_v<V>(p.h + row * p.ldh + c, y + i * V);
      }
    }
  }
}

// A group's rows: every gridDim * groups-th one, or (grouped gates) the
// slabs it owns, each within one gate row.  The parameter gradients of a
// group's rows stay in its threads' registers (16 columns each) and are
// added over the CTA's groups, in group order, at the end; slabs of a
// grouped gate are written out as each one ends.
template <typename R, int V, int THREADS>
__global__ void __launch_bounds__(THREADS) block_norm_bwd_kernel(const NormParams p) {
  constexpr int NV = kCols / V;
  __shared__ float red_all[16][64];
  const int warp = threadIdx.x >> 5;
  const int grp = warp / p.warps, wig = warp - grp * p.warps;
  const int t = threadIdx.x - grp * p.warps * 32, nt = p.warps * 32;
  float* red = red_all[grp];
  int turn = 0;
  const float inv_d = 1.0f / static_cast<float>(p.D);
  const int worker = blockIdx.x * p.groups + grp, workers = gridDim.x * p.groups;
  const bool slabbed = p.gate_mode == MOE_GATE_GROUP && p.dgate != nullptr;
  float aw_o[kCols], aw_h[kCols], ag[kCols];
#pragma unroll
  for (int i = 0; i < kCols; ++i) aw_o[i] = aw_h[i] = ag[i] = 0.0f;

  auto do_row = [&](long long row) {
    const R* x = static_cast<const R*>(p.x) + row * p.ldx;
    float y[kCols], n[kCols], s[kCols];   // s: dy, then the gradient of y; n: o r_o
    const float r_o = (p.o && p.w_post) ? p.stats[row] : 1.0f;
    const float r_y = p.w_pre ? p.stats[p.T + row] : 0.0f;
    float d[kCols];
    float saz = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * V;
#pragma unroll
      for (int j = 0; j < V; ++j) y[i * V + j] = n[i * V + j] = s[i * V + j] = d[i * V + j] = 0.0f;
      if (c < p.D) {
        load_v<V>(x + c, y + i * V);
        if (p.o) load_v<V>(p.o + row * p.ldo + c, n + i * V);
        if (p.dy) load_v<V>(static_cast<const R*>(p.dy) + row * p.lddy + c, s + i * V);
        if (p.w_pre) load_v<V>(p.dh + row * p.lddh + c, d + i * V);
      }
    }
    if (p.w_pre) {
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * V;
        if (c < p.D) {
          float w[V], g[V], wh[V];
          weight_v<V>(p, p.w_pre, c, wh);
          if (p.o) {
            weight_v<V>(p, p.w_post, c, w);
            gate_v<V>(p, row, c, g);
          }
#pragma unroll
          for (int j = 0; j < V; ++j) {
            const int k = i * V + j;
            float yy = p.alpha * y[k];
            if (p.o) yy = fmaf(p.beta, g[j] * (n[k] * r_o * w[j]), yy);
            const float z = yy * r_y;
            aw_h[k] = fmaf(d[k], z, aw_h[k]);
            const float a = d[k] * wh[j];
            saz = fmaf(a, z, saz);
            d[k] = a;
            y[k] = z;
          }
        }
      }
      const float m = group_sum(saz, red, p.warps, wig, 1 + grp, turn) * inv_d;
#pragma unroll
      for (int k = 0; k < kCols; ++k) s[k] = fmaf(r_y, d[k] - y[k] * m, s[k]);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * V;
      if (c < p.D && p.dx) {
        float v[V];
#pragma unroll
        for (int j = 0; j < V; ++j) v[j] = p.alpha * s[i * V + j];
        store_v<V>(static_cast<R*>(p.dx) + row * p.lddx + c, v);
      }
    }
    if (!p.o) return;
    float sbn = 0.0f, sg = 0.0f;
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * V;
      if (c < p.D) {
        float w[V], g[V];
        weight_v<V>(p, p.w_post, c, w);
        gate_v<V>(p, row, c, g);
#pragma unroll
        for (int j = 0; j < V; ++j) {
          const int k = i * V + j;
          const float nn = n[k] * r_o, bs = p.beta * s[k];
          const float dg = bs * nn * w[j];
          ag[k] += dg;
          sg += dg;
          const float bg = bs * g[j];
          aw_o[k] = fmaf(bg, nn, aw_o[k]);
          const float b = bg * w[j];
          sbn = fmaf(b, nn, sbn);
          s[k] = b;
          n[k] = nn;
        }
      }
    }
    if (p.gate_mode == MOE_GATE_TOKEN && p.dgate) {
      sg = group_sum(sg, red, p.warps, wig, 1 + grp, turn);
      if (t == 0) store_param<1>(p.dgate, p.gate_f32, row, &sg);
    }
    if (p.w_post) {
      const float m = group_sum(sbn, red, p.warps, wig, 1 + grp, turn) * inv_d;
#pragma unroll
      for (int k = 0; k < kCols; ++k) s[k] = r_o * (s[k] - n[k] * m);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int c = (t + i * nt) * V;
      if (c < p.D) store_v<V>(p.do_ + row * p.lddo + c, s + i * V);
    }
  };

  if (!slabbed) {
    for (long long row = worker; row < p.T; row += workers) do_row(row);
  } else {
    for (long long sl = worker; sl < p.slabs; sl += workers) {
      const int g = static_cast<int>(sl / p.slabs_per_group), j = static_cast<int>(sl - static_cast<long long>(g) * p.slabs_per_group);
      const int r0 = static_cast<int>(static_cast<long long>(p.rows_per_group) * j / p.slabs_per_group);
      const int r1 = static_cast<int>(static_cast<long long>(p.rows_per_group) * (j + 1) / p.slabs_per_group);
      for (int r = r0; r < r1; ++r) do_row(static_cast<long long>(g) * p.rows_per_group + r);
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int c = (t + i * nt) * V;
        if (c < p.D) {
          if (p.slabs_per_group == 1) store_param<V>(p.dgate, p.gate_f32, static_cast<long long>(g) * p.D + c, ag + i * V);
          else store_v<V>(p.gate_partial + sl * p.D + c, ag + i * V);
        }
#pragma unroll
        for (int k = 0; k < V; ++k) ag[i * V + k] = 0.0f;
      }
    }
  }
  // the CTA's parameter gradients, groups in order
  extern __shared__ float acc[];   // [D] per array when groups > 1
  const bool want[3] = {p.o != nullptr && p.w_post != nullptr, p.w_pre != nullptr,
                        p.gate_mode == MOE_GATE_CHANNEL && p.dgate != nullptr};
#pragma unroll
  for (int a = 0; a < 3; ++a) {
    if (!want[a]) continue;
    float* out = p.partial + (static_cast<long long>(a) * gridDim.x + blockIdx.x) * p.D;
    float* v = a == 0 ? aw_o : (a == 1 ? aw_h : ag);
    for (int g = 0; g < p.groups; ++g) {
      if (g == grp) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int c = (t + i * nt) * V;
          if (c < p.D) {
#pragma unroll
            for (int j = 0; j < V; ++j) {
              const float b = v[i * V + j] + (g > 0 ? acc[c + j] : 0.0f);
              if (g + 1 < p.groups) acc[c + j] = b;
              else out[c + j] = b;
            }
          }
        }
      }
      if (p.groups > 1) __syncthreads();
    }
  }
}

// out[c] = sum over r of in[r][c] for `rows` partial rows, in a fixed order:
// eight interleaved sums a column, then those in order.
__global__ void __launch_bounds__(256) column_sum_kernel(const float* __restrict__ in, int rows, int D, void* out0,
                                                         void* out1, void* out2, int f32_2) {
  __shared__ float part[8][33];
  const int a = blockIdx.y;
  void* out = a == 0 ? out0 : (a == 1 ? out1 : out2);
  if (out == nullptr) return;
  const int cx = threadIdx.x & 31, ry = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + cx;
  float s = 0.0f;
  if (c < D) {
    const float* p = in + static_cast<long long>(a) * rows * D + c;
#pragma unroll 8
    for (int r = ry; r < rows; r += 8) s += p[static_cast<long long>(r) * D];
  }
  part[ry][cx] = s;
  __syncthreads();
  if (ry == 0 && c < D) {
    for (int k = 1; k < 8; ++k) s += part[k][cx];
    store_param<1>(out, a == 2 ? f32_2 : 1, c, &s);
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
  store_param<1>(dgate, f32, static_cast<long long>(blockIdx.y) * D + c, &s);
}

// ------------------------------------------------------------------- host

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

struct Shape {
  int warps, groups, threads;
};

Shape shape_of(int D) {
  Shape s;
  s.warps = (D + kWarpCols - 1) / kWarpCols;
  s.groups = s.warps >= 8 ? 1 : 16 / s.warps;
  if (s.groups > 15) s.groups = 15;   // named barriers 1 .. 15
  s.threads = s.warps * s.groups * 32;
  return s;
}

template <typename R, int THREADS>
void launch_fwd(bool vec, int ctas, const Shape& s, const NormParams& p, cudaStream_t stream) {
  if (vec) block_norm_fwd_kernel<R, 8, THREADS><<<ctas, s.threads, 0, stream>>>(p);
  else block_norm_fwd_kernel<R, 1, THREADS><<<ctas, s.threads, 0, stream>>>(p);
}

template <typename R, int THREADS>
void launch_bwd(bool vec, int ctas, const Shape& s, size_t smem, const NormParams& p, cudaStream_t stream) {
  if (vec) block_norm_bwd_kernel<R, 8, THREADS><<<ctas, s.threads, smem, stream>>>(p);
  else block_norm_bwd_kernel<R, 1, THREADS><<<ctas, s.threads, smem, stream>>>(p);
}

int backward_ctas(const Shape& s, int T, int sms) {
  const int need = (T + s.groups - 1) / s.groups;
  return need < sms ? need : sms;
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

NormParams common_params(const moe_block_norm_config* c, const void* x, const void* branch, const void* gate,
                         const void* w_post, const void* w_pre) {
  NormParams p{};
  p.T = c->tokens;
  p.D = c->d_model;
  p.x = x;
  p.o = static_cast<const __nv_bfloat16*>(branch);
  p.gate = gate;
  p.w_post = branch ? w_post : nullptr;
  p.w_pre = w_pre;
  auto ld = [&](int64_t v) { return v ? static_cast<long long>(v) : static_cast<long long>(c->d_model); };
  p.ldx = ld(c->x_stride);
  p.ldo = ld(c->branch_stride);
  p.ldy = p.lddy = ld(c->y_stride);
  p.ldh = p.lddh = ld(c->h_stride);
  p.lddx = p.lddo = c->d_model;
  p.gate_mode = branch ? c->gate_mode : MOE_GATE_NONE;
  p.rows_per_group = p.gate_mode == MOE_GATE_GROUP ? c->tokens / c->gate_rows : 1;
  if (p.rows_per_group < 1) p.rows_per_group = 1;
  p.params_f32 = c->weight_type == MOE_TYPE_FP32;
  p.gate_f32 = c->gate_type == MOE_TYPE_FP32;
  p.alpha = c->residual_scale;
  p.beta = c->branch_scale;
  p.eps = c->eps;
  p.offset = c->weight_offset;
  return p;
}

bool vector_rows(const NormParams& p) {
  return p.D % 8 == 0 && p.ldx % 8 == 0 && p.ldo % 8 == 0 && p.ldy % 8 == 0 && p.ldh % 8 == 0 && p.lddy % 8 == 0 &&
         p.lddh % 8 == 0 && p.lddx % 8 == 0 && p.lddo % 8 == 0;
}

int device_sms() {
  static PerDeviceOnce once;
  static int sms[kMaxDevices];
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const cudaError_t e = once.once([&] { return cudaDeviceGetAttribute(&sms[dev], cudaDevAttrMultiProcessorCount, dev); });
  return e == cudaSuccess ? sms[dev] : 0;
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
  if (!branch && (gate || post_weight)) return MOE_ERR_INVALID_ARG;
  if (branch && (gate != nullptr) != (cfg->gate_mode != MOE_GATE_NONE)) return MOE_ERR_INVALID_ARG;
  if ((pre_weight != nullptr) != (h != nullptr)) return MOE_ERR_INVALID_ARG;
  if (cfg->tokens == 0) return MOE_OK;
  if (!x || (!y && !h)) return MOE_ERR_INVALID_ARG;
  for (const void* q : {x, branch, gate, post_weight, pre_weight, static_cast<const void*>(y),
                        static_cast<const void*>(h), static_cast<const void*>(stats)})
    if (!aligned16(q)) return MOE_ERR_INVALID_ARG;
  NormParams p = common_params(cfg, x, branch, gate, post_weight, pre_weight);
  p.y = y;
  p.h = static_cast<__nv_bfloat16*>(h);
  p.stats = stats;
  const Shape s = shape_of(p.D);
  p.warps = s.warps;
  p.groups = s.groups;
  const int sms = device_sms();
  if (sms <= 0) return MOE_ERR_CUDA;
  const int ctas = (p.T + s.groups - 1) / s.groups;
  const bool vec = vector_rows(p);
  const bool bf = cfg->residual_type == MOE_TYPE_BF16;
  if (s.threads <= 512) bf ? launch_fwd<__nv_bfloat16, 512>(vec, ctas, s, p, stream) : launch_fwd<float, 512>(vec, ctas, s, p, stream);
  else bf ? launch_fwd<__nv_bfloat16, 1024>(vec, ctas, s, p, stream) : launch_fwd<float, 1024>(vec, ctas, s, p, stream);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

size_t moe_block_norm_workspace_bytes(const moe_block_norm_config* cfg) {
  if (!config_ok(cfg) || cfg->d_model > kMaxCols) return 0;
  const int sms = device_sms();
  if (sms <= 0) return 0;
  const Shape s = shape_of(cfg->d_model);
  const size_t ctas = static_cast<size_t>(backward_ctas(s, cfg->tokens, sms));
  size_t rows = 3 * ctas;
  if (cfg->gate_mode == MOE_GATE_GROUP) rows += ctas * s.groups + 1;   // slab partials, when a gate row has several
  return (rows * static_cast<size_t>(cfg->d_model) * sizeof(float) + 255) / 256 * 256 + 256;
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
  const int T = cfg->tokens, D = cfg->d_model;
  if (T == 0) {   // no rows: the parameters' gradients are zero
    auto zero = [&](void* q, size_t n) { return q ? cudaMemsetAsync(q, 0, n, stream) : cudaSuccess; };
    const size_t gsz = (cfg->gate_type == MOE_TYPE_FP32 ? 4 : 2);
    const size_t grows = cfg->gate_mode == MOE_GATE_CHANNEL ? 1 : (cfg->gate_mode == MOE_GATE_GROUP ? cfg->gate_rows : 0);
    if (zero(dpost_weight, sizeof(float) * D) != cudaSuccess || zero(dpre_weight, sizeof(float) * D) != cudaSuccess ||
        zero(grows ? dgate : nullptr, grows * D * gsz) != cudaSuccess)
      return MOE_ERR_CUDA;
    return MOE_OK;
  }
  if (!x || ((post_weight || pre_weight) && !stats)) return MOE_ERR_INVALID_ARG;
  const size_t need = moe_block_norm_workspace_bytes(cfg);
  if (need == 0) return MOE_ERR_CUDA;
  if (!workspace || workspace_bytes < need) return MOE_ERR_CAPACITY;
  const int sms = device_sms();
  NormParams p = common_params(cfg, x, branch, gate, post_weight, pre_weight);
  p.stats = const_cast<float*>(stats);
  p.dy = dy;
  p.dh = static_cast<const __nv_bfloat16*>(dh);
  p.dx = dx;
  p.do_ = static_cast<__nv_bfloat16*>(dbranch);
  p.dgate = dgate;
  const Shape s = shape_of(D);
  p.warps = s.warps;
  p.groups = s.groups;
  const int ctas = backward_ctas(s, T, sms);
  p.partial = static_cast<float*>(workspace);
  p.gate_partial = p.partial + 3ll * ctas * D;
  if (p.gate_mode == MOE_GATE_GROUP) {
    const int workers = ctas * s.groups;
    int per = workers / cfg->gate_rows;
    if (per < 1) per = 1;
    if (per > p.rows_per_group) per = p.rows_per_group;
    p.slabs_per_group = per;
    p.slabs = per * cfg->gate_rows;
  }
  const bool vec = vector_rows(p);
  const size_t smem = s.groups > 1 ? static_cast<size_t>(D) * sizeof(float) : 0;
  const bool bf = cfg->residual_type == MOE_TYPE_BF16;
  if (s.threads <= 512) bf ? launch_bwd<__nv_bfloat16, 512>(vec, ctas, s, smem, p, stream) : launch_bwd<float, 512>(vec, ctas, s, smem, p, stream);
  else bf ? launch_bwd<__nv_bfloat16, 1024>(vec, ctas, s, smem, p, stream) : launch_bwd<float, 1024>(vec, ctas, s, smem, p, stream);
  if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  void* channel = p.gate_mode == MOE_GATE_CHANNEL ? dgate : nullptr;
  if (dpost_weight || dpre_weight || channel) {
    column_sum_kernel<<<dim3((D + 31) / 32, 3), 256, 0, stream>>>(p.partial, ctas, D, dpost_weight, dpre_weight, channel,
                                                                  p.gate_f32);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  }
  if (p.gate_mode == MOE_GATE_GROUP && p.slabs_per_group > 1) {
    gate_slab_sum_kernel<<<dim3((D + 255) / 256, cfg->gate_rows), 256, 0, stream>>>(p.gate_partial, p.slabs_per_group, D,
                                                                                    dgate, p.gate_f32);
    if (cudaGetLastError() != cudaSuccess) return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

}  // extern "C"
