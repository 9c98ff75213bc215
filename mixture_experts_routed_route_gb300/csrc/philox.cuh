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
// time, 2.5 wide products an element, which take the SMs 29 us for the 16384 x
// 7168 elements that stream from HBM in 69 (BF16).  With 32 bits it would be five.
#pragma once

#include "common.cuh"

namespace moe {

struct DropParams {
  const long long* rng;   // [seed, step] on the device; NULL: no dropout
  uint32_t site;
  uint32_t threshold;     // p 2^16, rounded: 0 .. 65536
  uint32_t least;         // in both halves: the least 16 bits that are kept
  uint32_t low, high;     // 0xFFFF, 0xFFFF0000; zeros where everything is dropped
  float scale;            // 2^16 / (2^16 - threshold); 0 where everything is dropped
};

// Host: fill from p; false if p is no probability.
inline bool drop_params(DropParams* d, const void* rng, double p, uint32_t site) {
  if (!(p >= 0.0 && p <= 1.0)) return false;
  d->threshold = static_cast<uint32_t>(p * 65536.0 + 0.5);
  d->least = (d->threshold < 65535u ? d->threshold : 65535u) * 0x10001u;
  d->low = d->threshold < 65536u ? 0x0000FFFFu : 0u;
  d->high = d->threshold < 65536u ? 0xFFFF0000u : 0u;
  d->rng = d->threshold ? static_cast<const long long*>(rng) : nullptr;
  d->site = site;
  d->scale = d->threshold >= 65536u ? 0.0f : 65536.0f / static_cast<float>(65536u - d->threshold);
  return true;
}

// The generator's keys, and what of its first round is the same for every
// element of a call.  KEEP: the ten rounds' keys stay in registers, 18 more,
// instead of being added up for each block.
template <bool KEEP>
struct PhiloxKey {
  uint32_t k0, k1;        // of the first round
  uint32_t h1, l1;        // the first round's product with the site
  uint32_t step;
  uint32_t kept0[KEEP ? 10 : 1], kept1[KEEP ? 10 : 1];
  __device__ __forceinline__ uint32_t key0(int r) const { return KEEP ? kept0[r] : k0 + r * 0x9E3779B9u; }
  __device__ __forceinline__ uint32_t key1(int r) const { return KEEP ? kept1[r] : k1 + r * 0xBB67AE85u; }
};

template <bool KEEP>
__device__ __forceinline__ PhiloxKey<KEEP> philox_key(const DropParams& d) {
  const long long seed = d.rng[0];
  PhiloxKey<KEEP> k;
  k.k0 = static_cast<uint32_t>(seed);
  k.k1 = static_cast<uint32_t>(static_cast<unsigned long long>(seed) >> 32);
#pragma unroll
  for (int r = 0; r < (KEEP ? 10 : 0); ++r) {
    k.kept0[r] = k.k0 + r * 0x9E3779B9u;
    k.kept1[r] = k.k1 + r * 0xBB67AE85u;
  }
  const unsigned long long b = static_cast<unsigned long long>(d.site) * 0xCD9E8D57u;
  k.h1 = static_cast<uint32_t>(b >> 32) ^ k.k0;
  k.l1 = static_cast<uint32_t>(b);
  k.step = static_cast<uint32_t>(d.rng[1]) ^ k.k1;
  return k;
}

// The block of counter (group, site, step).
template <bool KEEP>
__device__ __forceinline__ uint4 philox(const PhiloxKey<KEEP>& key, unsigned long long group) {
  unsigned long long a = static_cast<unsigned long long>(static_cast<uint32_t>(group)) * 0xD2511F53u, b;
  uint32_t c0 = key.h1 ^ static_cast<uint32_t>(group >> 32), c1 = key.l1;
  uint32_t c2 = static_cast<uint32_t>(a >> 32) ^ key.step, c3 = static_cast<uint32_t>(a);
#pragma unroll
  for (int r = 1; r < 10; ++r) {
    a = static_cast<unsigned long long>(c0) * 0xD2511F53u;
    b = static_cast<unsigned long long>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(b >> 32) ^ c1 ^ key.key0(r);
    c2 = static_cast<uint32_t>(a >> 32) ^ c3 ^ key.key1(r);
    c1 = static_cast<uint32_t>(b);
    c3 = static_cast<uint32_t>(a);
  }
  return make_uint4(c0, c1, c2, c3);
}

// The block's eight elements as four words of two: all ones in the half of an
// element that is kept, zeros in that of a dropped one.  One instruction
// compares both halves of a word.
__device__ __forceinline__ uint4 keep_words(const DropParams& d, const uint4& w) {
  const uint32_t in[4] = {w.x, w.y, w.z, w.w};
  uint32_t out[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    bool hi, lo;
    __vibmax_u16x2(in[j], d.least, &hi, &lo);
    out[j] = (lo ? d.low : 0u) | (hi ? d.high : 0u);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}
// Element j's half of them (j a constant).
__device__ __forceinline__ bool kept(const uint4& m, int j) {
  const uint32_t word = j < 2 ? m.x : j < 4 ? m.y : j < 6 ? m.z : m.w;
  return (word & ((j & 1) ? 0xFFFF0000u : 0x0000FFFFu)) != 0;
}

}  // namespace moe
