// What a query behind a sliding window sees, one bit a key.  Plain C++, so that it also runs on the host.
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define PA_WINDOW_FN __host__ __device__ __forceinline__
#else
#define PA_WINDOW_FN inline
#endif

namespace pa {

// First position of the window of the query at position `bound` (-1: of a row that sees nothing).
PA_WINDOW_FN int window_low(int bound, int window) { return bound < window ? 0 : bound - window + 1; }

// Keys k0 .. k0 + 31 that it sees: up to its own position, from `low` on or below the sinks' end.  (low is at least 0, so no
// difference of two positions leaves 32 bits.)
PA_WINDOW_FN uint32_t window_seen32(int bound, int low, int sinks, int k0) {
  const int nv = bound - k0 + 1, from = low > k0 ? low - k0 : 0, to = sinks > k0 ? sinks - k0 : 0;
  const uint32_t m = nv >= 32 ? 0xFFFFFFFFu : (nv <= 0 ? 0u : ((1u << nv) - 1u));
  return m & ((from < 32 ? 0xFFFFFFFFu << from : 0u) | (to < 32 ? (1u << to) - 1u : 0xFFFFFFFFu));
}

}  // namespace pa
