// Device helpers shared by the kernels of the paged key-value cache.
#pragma once

#include "nvfp4_device.h"
#include "paged_internal.h"

namespace nvfp4 {

__device__ __forceinline__ int clamp_int(int v, int lo, int hi) { return v < lo ? lo : (v > hi ? hi : v); }

// A load from a wave-uniform address that no kernel writes while this one runs: a scalar load.  (As a vector
// load its use would wait for every vector load issued before it, the prefetched keys and values among
// them.)
template <typename T>
__device__ __forceinline__ T scalar_load(const T* p) {
  return *reinterpret_cast<const __attribute__((address_space(4))) T*>(reinterpret_cast<uintptr_t>(p));
}

// Largest j in [0, n) with pred(j), for a predicate that holds on a prefix; -1 if it holds nowhere.
// Called by whole wavefronts with uniform arguments: 64 probes a round, so one round of loads up
// to 64 entries and two up to 4096.
template <typename Pred>
__device__ __forceinline__ int wave_search(int n, Pred pred) {
  const int lane = threadIdx.x & 63;
  int lo = 0, cnt = n;
  while (true) {
    const int stride = (cnt + 63) >> 6;
    const int j = lane * stride;
    const bool in = j < cnt && pred(lo + j);
    const int k = __builtin_popcountll(__builtin_amdgcn_ballot_w64(in));
    if (k == 0) return lo - 1;       // only in the first round: later rounds start on an entry that holds
    lo += (k - 1) * stride;
    if (stride == 1) return lo;
    cnt = cnt - (k - 1) * stride < stride ? cnt - (k - 1) * stride : stride;
  }
}

}  // namespace nvfp4
