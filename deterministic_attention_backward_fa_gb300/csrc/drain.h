// Waiting on the way out, in plain C++ so that it can be tested on the host too.
#pragma once

#include <cstdint>

#ifdef __CUDACC__
#define DASH_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define DASH_HOST_DEVICE inline
#endif

namespace dash {

// Waits until done(i) holds for each i < n, one after the other, for `limit` of
// the clock in all: after an abort several of them may never hold.
template <class Done, class Clock>
DASH_HOST_DEVICE void drain_all(int n, Done done, Clock now, uint64_t limit) {
  const uint64_t t0 = now();
  for (int i = 0; i < n; ++i)
    while (!done(i))
      if (now() - t0 > limit) return;
}

}  // namespace dash
