// Host-side helpers of the paged-cache entry points.
#pragma once
#include <cuda_runtime.h>

#include <cstdint>

namespace smla {

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

}  // namespace smla
