// The dropout mask: a counter-based generator, so that the backward pass (or
// any other kernel) draws the same mask again and none is stored.
//
// Philox4x32 with ten rounds (Salmon, Moraes, Dror, Shaw, "Parallel random
// numbers: as easy as 1, 2, 3", 2011): a bijection of 128-bit counters under a
// 64-bit key, two 32 x 32 -> 64 bit products a round.  Element e = t D + d of
// the [T, D] tensor takes 16 bits of the block with counter (e / 8 low word,
// e / 8 high word, site, step): half e % 2 of word (e % 8) / 2.  It is kept if
// those 16 bits, as a number, are at least the threshold p 2^16.
// 16 bits an element: one block serves the 8 elements a thread handles at a
// time, 2.5 wide products an element.  With 32 bits it would be five, about as
// many as the SMs issue while the elements stream from HBM.
#pragma once

#include "common.cuh"

namespace moe {

struct DropParams {
  const long long* rng;   // [seed, step] on the device; NULL: no dropout
  uint32_t site;
  uint32_t threshold;     // p 2^16, rounded: 0 .. 65536
  float scale;            // 2^16 / (2^16 - threshold); 0 where everything is dropped
};

// Host: fill from p; false if p is no probability.
inline bool drop_params(DropParams* d, const void* rng, double p, uint32_t site) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  d->threshold = static_cast<uint32_t>(p * 65536.0 + 0.5);
  d->rng = d->threshold ? static_cast<const long long*>(rng) : nullptr;
  d->site = site;
  d->scale = d->threshold >= 65536u ? 0.0f : 65536.0f / static_cast<float>(65536u - d->threshold);
  return true;
}

struct PhiloxKey {
  uint32_t k0, k1, site, step;
};

__device__ __forceinline__ PhiloxKey philox_key(const DropParams& d) {
  const long long seed = d.rng[0], step = d.rng[1];
  return {static_cast<uint32_t>(seed), static_cast<uint32_t>(static_cast<unsigned long long>(seed) >> 32), d.site,
          static_cast<uint32_t>(step)};
}

// The block of counter (group, site, step).
__device__ __forceinline__ uint4 philox(const PhiloxKey& key, unsigned long long group) {
  uint32_t c0 = static_cast<uint32_t>(group), c1 = static_cast<uint32_t>(group >> 32), c2 = key.site, c3 = key.step;
  uint32_t k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const unsigned long long a = static_cast<unsigned long long>(c0) * 0xD2511F53u;
    const unsigned long long b = static_cast<unsigned long long>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Whether element j of the block's eight is kept (j a constant).
__device__ __forceinline__ bool kept(const uint4& w, int j, uint32_t threshold) {
  const uint32_t word = j < 2 ? w.x : j < 4 ? w.y : j < 6 ? w.z : w.w;
  return ((j & 1) ? word >> 16 : word & 0xFFFFu) >= threshold;
}

}  // namespace moe
