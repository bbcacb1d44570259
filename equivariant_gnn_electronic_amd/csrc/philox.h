// Counter-based random decisions shared by the dropout operators.
//
// Philox4x32-10 (Salmon, Moraes, Dror, Shaw, "Parallel random numbers: as easy
// as 1, 2, 3", SC 2011): ten rounds of two 32x32->64 products.  Key = the
// 64-bit seed; counter = (low and high word of i/8, step, site) for decision
// i, so one call decides eight consecutive i: 16-bit draw i%8, the low half of
// each word first.  Decision i keeps iff its draw >= t, t = round(65536 p).
// Sixteen bits a draw because the ten rounds' integer products, not memory,
// would bound a mask that is spent on one element;
// they quantise p to 1/65536, and the factor 65536/(65536 - t) is that of the
// quantised p, so the expectation is exact.
#pragma once

#include "common.h"

namespace egnn {

struct Drop {
  const uint64_t *rng;  // device [2]: seed, step (low 32 bits); null when t == 0
  uint32_t site;
  uint32_t t;      // 0: keep everything
  float factor;    // 65536 / (65536 - t)
};

// threshold of p, or -1 for a p that is not in [0, 1) after rounding
inline int drop_threshold(double p) {
  if (!(p >= 0.0) || !(p < 1.0)) return -1;
  const int t = static_cast<int>(p * 65536.0 + 0.5);
  return t < 65536 ? t : -1;
}

inline Drop make_drop(const uint64_t *rng, uint32_t site, int t) {
  return Drop{rng, site, static_cast<uint32_t>(t), 65536.0f / static_cast<float>(65536 - t)};
}

struct DropKey {
  uint32_t k0, k1, step, site;
};

__device__ inline DropKey drop_key(const Drop &d) {
  const uint64_t seed = d.rng[0], step = d.rng[1];
  return DropKey{static_cast<uint32_t>(seed), static_cast<uint32_t>(seed >> 32), static_cast<uint32_t>(step), d.site};
}

__device__ inline uint4 philox4x32(uint64_t j, const DropKey &k) {
  uint32_t c0 = static_cast<uint32_t>(j), c1 = static_cast<uint32_t>(j >> 32), c2 = k.step, c3 = k.site;
  uint32_t k0 = k.k0, k1 = k.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(c0) * 0xD2511F53u;
    const uint64_t p1 = static_cast<uint64_t>(c2) * 0xCD9E8D57u;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c1 = static_cast<uint32_t>(p1);
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// draw u (0..7) of one call
__device__ inline uint32_t drop_draw(const uint4 &w, int u) {
  const uint32_t word = (u & 4) ? ((u & 2) ? w.w : w.z) : ((u & 2) ? w.y : w.x);
  return (u & 1) ? word >> 16 : word & 0xFFFFu;
}

// 0 or the factor, for one decision
__device__ inline float drop_one(int64_t i, const Drop &d, const DropKey &k) {
  const uint4 w = philox4x32(static_cast<uint64_t>(i) >> 3, k);
  return drop_draw(w, static_cast<int>(i & 7)) >= d.t ? d.factor : 0.0f;
}

}  // namespace egnn
