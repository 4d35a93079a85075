// Host-side check of tensor ranges.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace moonep {

// Whether two byte ranges share memory.
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na > 0 && nb > 0 && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

struct Range {
  const void* at;
  int64_t bytes;
};

// Whether a written range shares memory with a read one or another written one:
// a workgroup would write what another has yet to read.
template <size_t W, size_t R>
inline bool clash(const Range (&written)[W], const Range (&read)[R]) {
  for (size_t i = 0; i < W; ++i) {
    for (const Range& r : read)
      if (overlap(written[i].at, written[i].bytes, r.at, r.bytes)) return true;
    for (size_t j = 0; j < i; ++j)
      if (overlap(written[i].at, written[i].bytes, written[j].at, written[j].bytes)) return true;
  }
  return false;
}

}  // namespace moonep
