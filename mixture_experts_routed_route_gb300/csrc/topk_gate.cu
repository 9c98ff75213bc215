// The router's choice: top_k experts a token from its logits, their scores,
// and the gradient of the logits (moe_topk_gate_forward / _backward).
//
// key_e = logit_e + bias_e (one FP32 rounding; the bias steers the choice
// only).  The K largest keys are taken, equal keys by ascending expert, keys
// of -inf never; places without an expert get id -1 and score 0, the layer's
// inactive route.  With scale c, over l = the logits:
//   softmax                s_k = c exp(l_k) / sum over all experts
//   softmax, renormalised  s_k = c exp(l_k) / sum over the chosen
//   sigmoid                s_k = c sig(l_k)
//   sigmoid, renormalised  s_k = c sig(l_k) / (sum over the chosen + 1e-20)
// Gradients, with d_k = c ds_k and v_k the unscaled scores:
//   softmax                dl_e = [e chosen] v_e d_e - p_e sum_k v_k d_k
//   softmax, renormalised  dl_k = v_k (d_k - sum_j v_j d_j), 0 elsewhere
//   sigmoid                dl_k = d_k sig(l_k) sig(-l_k), 0 elsewhere;
//   renormalised           d_k -> (d_k - sum_j v_j d_j) / (sum + 1e-20) first
// A row with a NaN or +inf logit has no choice: ids -1, scores NaN (and a
// NaN gradient), so the fault shows instead of routing somewhere.
//
// One warp a token; lane i holds the logits of experts i, i + 32, ...  Keys
// are compared as their order-preserving 32-bit images.  The choice takes two
// short steps instead of top_k passes over all keys: the top_k-th largest of
// the 32 lanes' own maxima is a bound that at least top_k keys reach and few
// others do (a round of redux.sync a distinct maximum); those that reach it
// are gathered, one a lane, and each counts the ones before it.  Rows where
// more than 32 keys reach the bound (ties) take them one by one.  What bounds
// the pass is instruction issue, not the bytes: 16384 x 384, top 8, went from
// 26 us with one pass over the lanes' keys per choice to 15.6 us (floor 3.9),
// about 700 instructions a token (sigmoid scores with a bias; a softmax over
// all experts takes as long).  A grid that stays and loads a token ahead took 16.5 to 18.9 us
// (more registers, fewer warps); 65536 x 64, top 6, takes 24 us, one token 3.4.
// The backward reads and writes whole rows once: 4096 x 384 7.4 us (1.7 TB/s,
// mostly the latency of one launch and one row), 16384 x 384 over all experts
// 18.7 us (2.7 TB/s), top 8 renormalised softmax 16.8, sigmoid 20.6 (these read
// the row for its NaN or +inf alone).  From eight logits a lane on the row is
// an array in local memory, indexed by the chosen terms that are added to it.
#include "kernels.cuh"
#include "moe_gb300.h"

namespace moe {

namespace {

constexpr int kGateThreads = 256;
constexpr float kSigmoidEps = 1e-20f;

struct GateParams {
  int T, E, K;
  const void* logits;   // [T, ld]
  long long ld;
  const float* bias;    // [E] or NULL
  int sigmoid, renorm;
  float scale;
  int* ids;             // [T, K]
  float* scores;        // [T, K] (backward: gradient of the scores)
  void* dlogits;        // [T, E]
};

// Unsigned image of a float with the same order (-0 like +0 beforehand).
__device__ __forceinline__ uint32_t order_of(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
  return u ^ ((u >> 31) ? 0xFFFFFFFFu : 0x80000000u);
}
constexpr uint32_t kOrderNegInf = 0x007FFFFFu;   // order_of(-inf)

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

__device__ __forceinline__ float to_f(float v) { return v; }
__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void put(float* p, float v) { *p = v; }
__device__ __forceinline__ void put(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// L = experts per lane (ceil(E / 32) rounded up to the instance).
template <typename X, int L>
__global__ void __launch_bounds__(kGateThreads) topk_gate_fwd_kernel(const GateParams p) {
  const int lane = threadIdx.x & 31;
  __shared__ uint2 lists[kGateThreads / 32][32];
  uint2* list = lists[threadIdx.x >> 5];
  const long long t = static_cast<long long>(blockIdx.x) * (kGateThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const X* row = static_cast<const X*>(p.logits) + t * p.ld;
  float l[L];
  uint32_t key[L];
  bool bad = false;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    l[i] = -INFINITY;
    if (e < p.E) l[i] = to_f(row[e]);
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    const float b = (p.bias && e < p.E) ? l[i] + p.bias[e] : l[i];
    key[i] = e < p.E ? order_of(b) : 0u;
    bad |= !(l[i] < INFINITY && b < INFINITY);
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  // the K choices: lane k keeps the k-th
  int my_id = -1;
  float my_l = 0.0f;
  if (!bad) {
    uint32_t own = key[0];
#pragma unroll
    for (int i = 1; i < L; ++i) own = max(own, key[i]);
    // the bound: the K-th largest lane maximum (all keys above -inf, if fewer)
    uint32_t bound = kOrderNegInf + 1, left = own;
    for (int found = 0; found < p.K;) {
      const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, left);
      if (top <= kOrderNegInf) {
        bound = kOrderNegInf + 1;
        break;
      }
      bound = top;
      found += __popc(__ballot_sync(0xFFFFFFFFu, left == top));
      if (left == top) left = 0u;
    }
    // the keys that reach it, in ascending expert order
    int n = 0;
#pragma unroll
    for (int i = 0; i < L; ++i) {
      const uint32_t reach = __ballot_sync(0xFFFFFFFFu, key[i] >= bound);
      const int at = n + __popc(reach & ((1u << lane) - 1u));
      if (key[i] >= bound && at < 32) list[at] = make_uint2(key[i], static_cast<uint32_t>(lane + 32 * i));
      n += __popc(reach);
    }
    __syncwarp();
    if (n <= 32) {
      const uint2 c = lane < n ? list[lane] : make_uint2(0u, 0u);
      int rank = 0;
      for (int j = 0; j < n; ++j) {
        const uint32_t k = __shfl_sync(0xFFFFFFFFu, c.x, j);
        rank += k > c.x || (k == c.x && j < lane);
      }
      __syncwarp();
      if (lane < n && rank < 32) list[rank] = c;   // in the order of choice
      __syncwarp();
      if (lane < min(n, p.K)) {
        my_id = static_cast<int>(list[lane].y);
        my_l = to_f(row[my_id]);
      }
    } else {
      uint32_t best = 0;
      int at = 0;
      auto rescan = [&] {
        best = key[0];
        at = 0;
#pragma unroll
        for (int i = 1; i < L; ++i)
          if (key[i] > best) best = key[i], at = i;
      };
      rescan();
      for (int k = 0; k < p.K; ++k) {
        const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
        if (top <= kOrderNegInf) break;
        const int e = lane + 32 * at;
        const int who = __reduce_min_sync(0xFFFFFFFFu, best == top ? e : 0x7FFFFFFF);
        if (who == e && best == top) {
#pragma unroll
          for (int i = 0; i < L; ++i)
            if (i == at) key[i] = 0u;
          rescan();
        }
        if (lane == k) my_id = who;
      }
      if (my_id >= 0) my_l = to_f(row[my_id]);
    }
  }
  const bool on = my_id >= 0;
  float s = 0.0f;
  if (p.sigmoid) {
    s = on ? 1.0f / (1.0f + expf(-my_l)) : 0.0f;
    if (p.renorm) s = s / (warp_sum(s) + kSigmoidEps);
  } else if (p.renorm) {
    const float m = warp_max(on ? my_l : -INFINITY);
    s = on ? expf(my_l - m) : 0.0f;
    const float sum = warp_sum(s);
    if (on) s = s / sum;
  } else {
    float m = l[0];
#pragma unroll
    for (int i = 1; i < L; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < L; ++i) sum += expf(l[i] - m);
    sum = warp_sum(sum);
    if (on) s = expf(my_l - m) / sum;
  }
  if (lane < p.K) {
    const long long o = t * p.K + lane;
    p.ids[o] = my_id;
    p.scores[o] = bad ? NAN : (on ? s * p.scale : 0.0f);
  }
}

template <typename X, int L>
__global__ void __launch_bounds__(kGateThreads) topk_gate_bwd_kernel(const GateParams p) {
  const int lane = threadIdx.x & 31;
  const bool dense = !p.sigmoid && !p.renorm;
  const long long t = static_cast<long long>(blockIdx.x) * (kGateThreads / 32) + (threadIdx.x >> 5);
  if (t >= p.T) return;
  const X* row = static_cast<const X*>(p.logits) + t * p.ld;
  X* out = static_cast<X*>(p.dlogits) + t * p.E;
  int id = -1;
  float d = 0.0f;
  if (lane < p.K) {
    const long long o = t * p.K + lane;
    id = p.ids[o];
    if (id < 0 || id >= p.E) id = -1;   // a bad id is an inactive route
    if (id >= 0) d = p.scale * p.scores[o];
  }
  const bool on = id >= 0;
  float l[L];
  bool bad = false;
  float m = -INFINITY;
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    l[i] = -INFINITY;
    if (e < p.E) l[i] = to_f(row[e]);
    bad |= !(l[i] < INFINITY);
  }
  bad = __any_sync(0xFFFFFFFFu, bad);
  const float lk = on ? to_f(row[id]) : -INFINITY;
  float dl = 0.0f;
  if (p.sigmoid) {
    const float v = on ? 1.0f / (1.0f + expf(-lk)) : 0.0f;
    const float slope = on ? v / (1.0f + expf(lk)) : 0.0f;
    if (p.renorm) {
      const float sum = warp_sum(v) + kSigmoidEps;
      const float dot = warp_sum(d * (v / sum));
      dl = on ? (d - dot) / sum * slope : 0.0f;
    } else {
      dl = d * slope;
    }
  } else if (p.renorm) {
    const float top = warp_max(lk);
    const float v = on ? expf(lk - top) : 0.0f;
    const float sum = warp_sum(v);
    const float sv = on ? v / sum : 0.0f;
    const float dot = warp_sum(d * sv);
    dl = sv * d - sv * dot;
  } else {
#pragma unroll
    for (int i = 0; i < L; ++i) m = fmaxf(m, l[i]);
    m = warp_max(m);
    float sum = 0.0f;
    if (m > -INFINITY) {
#pragma unroll
      for (int i = 0; i < L; ++i) {
        l[i] = expf(l[i] - m);
        sum += l[i];
      }
    }
    sum = warp_sum(sum);
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const float pk = on ? expf(lk - m) * inv : 0.0f;
    const float dot = warp_sum(pk * d);
    dl = pk * d;
#pragma unroll
    for (int i = 0; i < L; ++i) l[i] = m > -INFINITY ? -(l[i] * inv) * dot : 0.0f;
  }
  if (!dense) {
#pragma unroll
    for (int i = 0; i < L; ++i) l[i] = 0.0f;
  }
  // add the chosen experts' own terms to the lanes that hold them
  for (int k = 0; k < p.K; ++k) {
    const int e = __shfl_sync(0xFFFFFFFFu, id, k);
    const float v = __shfl_sync(0xFFFFFFFFu, dl, k);
    if (e >= 0 && (e & 31) == lane) {
#pragma unroll
      for (int i = 0; i < L; ++i)
        if (i == (e >> 5)) l[i] += v;
    }
  }
#pragma unroll
  for (int i = 0; i < L; ++i) {
    const int e = lane + 32 * i;
    if (e < p.E) put(out + e, bad ? NAN : l[i]);
  }
}

template <typename X, int L>
void launch_gate(bool fwd, const GateParams& p, cudaStream_t stream) {
  const int per = kGateThreads / 32;
  const int ctas = (p.T - 1) / per + 1;
  if (fwd) topk_gate_fwd_kernel<X, L><<<ctas, kGateThreads, 0, stream>>>(p);
  else topk_gate_bwd_kernel<X, L><<<ctas, kGateThreads, 0, stream>>>(p);
}

template <typename X>
void launch_gate_l(bool fwd, const GateParams& p, cudaStream_t stream) {
  const int l = (p.E + 31) / 32;
  if (l <= 1) launch_gate<X, 1>(fwd, p, stream);
  else if (l <= 2) launch_gate<X, 2>(fwd, p, stream);
  else if (l <= 4) launch_gate<X, 4>(fwd, p, stream);
  else if (l <= 8) launch_gate<X, 8>(fwd, p, stream);
  else if (l <= 12) launch_gate<X, 12>(fwd, p, stream);
  else if (l <= 16) launch_gate<X, 16>(fwd, p, stream);
  else launch_gate<X, 32>(fwd, p, stream);
}

bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15) == 0; }

moe_status gate_call(bool fwd, const moe_topk_gate_config* c, const void* logits, const float* bias, int32_t* ids,
                     float* scores, void* dlogits, cudaStream_t stream) {
  if (!c || c->tokens < 0 || c->num_experts < 1 || c->num_experts > 1024) return MOE_ERR_INVALID_ARG;
  if (c->top_k < 1 || c->top_k > 32 || c->top_k > c->num_experts) return MOE_ERR_INVALID_ARG;
  if (c->logits_type != MOE_TYPE_BF16 && c->logits_type != MOE_TYPE_FP32) return MOE_ERR_INVALID_ARG;
  if (c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) return MOE_ERR_INVALID_ARG;
  if (c->logits_stride != 0 && c->logits_stride < c->num_experts) return MOE_ERR_INVALID_ARG;
  if (!(c->scale >= -3.0e38f && c->scale <= 3.0e38f)) return MOE_ERR_INVALID_ARG;
  if (c->tokens == 0) return MOE_OK;
  if (!logits || !ids || !scores || (!fwd && !dlogits)) return MOE_ERR_INVALID_ARG;
  if (!aligned16(logits) || !aligned16(bias) || !aligned16(ids) || !aligned16(scores) || !aligned16(dlogits))
    return MOE_ERR_INVALID_ARG;
  GateParams p{};
  p.T = c->tokens;
  p.E = c->num_experts;
  p.K = c->top_k;
  p.logits = logits;
  p.ld = c->logits_stride ? c->logits_stride : c->num_experts;
  p.bias = bias;
  p.sigmoid = c->score == MOE_SCORE_SIGMOID;
  p.renorm = c->renormalize != 0;
  p.scale = c->scale;
  p.ids = ids;
  p.scores = scores;
  p.dlogits = dlogits;
  if (c->logits_type == MOE_TYPE_FP32) launch_gate_l<float>(fwd, p, stream);
  else launch_gate_l<__nv_bfloat16>(fwd, p, stream);
  return cudaGetLastError() == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

moe_status moe_topk_gate_forward(const moe_topk_gate_config* cfg, const void* logits, const float* select_bias,
                                 int32_t* ids, float* scores, cudaStream_t stream) {
  return gate_call(true, cfg, logits, select_bias, ids, scores, nullptr, stream);
}

moe_status moe_topk_gate_backward(const moe_topk_gate_config* cfg, const void* logits, const int32_t* ids,
                                  const float* d_scores, void* d_logits, cudaStream_t stream) {
  return gate_call(false, cfg, logits, nullptr, const_cast<int32_t*>(ids), const_cast<float*>(d_scores), d_logits,
                   stream);
}

}  // extern "C"
