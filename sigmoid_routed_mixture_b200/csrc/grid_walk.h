// grid_walk.h -- the elements first, first + step, ... below n that one thread
// of a grid takes.  The index is 64-bit: with 32 bits it wraps where n is within
// one step of 2^31, and the walk goes on at negative indices.  (Plain C++, so
// that the host can walk it too.)
#pragma once

#include <stdint.h>

#ifdef __CUDACC__
#define SRM_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define SRM_HOST_DEVICE inline
#endif

namespace srm {

template <typename F>
SRM_HOST_DEVICE void grid_walk(int64_t first, int64_t step, int64_t n, F f) {
  for (int64_t i = first; i < n; i += step) f(static_cast<int>(i));
}

}  // namespace srm
