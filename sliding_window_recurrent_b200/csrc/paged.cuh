// What the kernels of the paged cache share: RoPE frequencies and page lookups.
#pragma once

#include <cmath>

#include "common.cuh"
#include "launchers.h"

namespace maglev {

// base^(-2c/hd), c < hd/2, formed once on the host in double.
struct RopeFreqs {
  double inv_freq[64];
};
inline RopeFreqs rope_freqs(int hd, double log2_base) {
  RopeFreqs r{};
  const double base = std::exp2(log2_base);
  for (int c = 0; c < hd / 2 && c < 64; ++c) r.inv_freq[c] = std::pow(base, -2.0 * c / hd);
  return r;
}

// cos and sin of p * theta: the product is formed and reduced to [-pi, pi] in
// double, so that positions up to 2^30 keep float accuracy.
__device__ __forceinline__ float2 rope_turn(int64_t p, double inv_freq) {
  double ang = (double)p * inv_freq;
  ang -= 6.283185307179586476925286766559 * rint(ang * 0.15915494309189533577);
  float2 r;
  sincosf((float)ang, &r.y, &r.x);
  return r;
}

inline int log2_of(int x) {  // of a power of two
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

}  // namespace maglev
