// What the kernels of the paged cache share: RoPE frequencies and page lookups.
#pragma once

#include <cmath>

#include "common.cuh"
#include "launchers.h"

namespace maglev {

// base^(-2c/hd) / (2 pi), c < hd/2: turns per position, formed once on the host.
struct RopeFreqs {
  double turns[64];
};
inline const RopeFreqs& rope_freqs(int hd, double log2_base) {
  // a thread's last table: 64 powers on the host cost as much as the launch
  static thread_local RopeFreqs r;
  static thread_local int last_hd = 0;
  static thread_local double last_base = 0;
  if (hd == last_hd && log2_base == last_base) return r;
  last_hd = hd;
  last_base = log2_base;
  const double base = std::exp2(log2_base);
  for (int c = 0; c < hd / 2 && c < 64; ++c)
    r.turns[c] = std::pow(base, -2.0 * c / hd) / 6.283185307179586476925286766559;
  return r;
}

// cos and sin of the angle of position p. Whole turns are dropped in double (the
// product is not rounded before), so that positions up to 2^30 keep float
// accuracy; sincospif then needs no range reduction of its own (a sincosf of
// the angle cost a lone warp 1.9 k cycles, this 0.4 k).
__device__ __forceinline__ float2 rope_turn(int64_t p, double turns) {
  const double x = (double)p, n = rint(x * turns);
  float2 r;
  sincospif(2.0f * (float)fma(x, turns, -n), &r.y, &r.x);
  return r;
}

inline int log2_of(int x) {  // of a power of two
  int n = 0;
  while ((1 << n) < x) ++n;
  return n;
}

// Launches a kernel whose blocks may be scheduled before the stream's last kernel
// has ended (programmatic dependent launch). Every thread of it calls
// wait_for_last() before it touches what earlier work reads or writes, and takes its
// pointers without __restrict__: the inputs may still be written while its first blocks
// wait, and const __restrict__ would promise that nothing writes them while it runs (loads
// through the read-only path, or from before the wait). Called one after another,
// without a graph, such calls follow each other 2 to 4 us sooner.
template <typename... Params, typename... Args>
cudaError_t launch_dependent(void (*kern)(Params...), dim3 blocks, unsigned threads, size_t smem, cudaStream_t st,
                             const Args&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = blocks;
  cfg.blockDim = dim3(threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, Params(args)...);
}
// Waits until the stream's last kernel has ended and its writes are visible.
__device__ __forceinline__ void wait_for_last() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
// The next kernel's blocks may be scheduled from here on (they wait for this one's end).
__device__ __forceinline__ void let_next_start() { asm volatile("griddepcontrol.launch_dependents;"); }

}  // namespace maglev
