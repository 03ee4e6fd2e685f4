// Host-side helpers of the paged-cache entry points.
#pragma once
#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>

namespace smla {

inline bool aligned_to(const void* p, uintptr_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + nb && y < x + na;
}

struct Span {
  const void* p;
  size_t n;
};

// Whether what a call writes overlaps one of its inputs, or other memory that it writes.
template <size_t N, size_t M>
inline bool any_overlap(const Span (&in)[N], const Span (&written)[M]) {
  for (size_t o = 0; o < M; ++o) {
    for (const Span& i : in)
      if (overlap(written[o].p, written[o].n, i.p, i.n)) return true;
    for (size_t u = o + 1; u < M; ++u)
      if (overlap(written[o].p, written[o].n, written[u].p, written[u].n)) return true;
  }
  return false;
}

}  // namespace smla
