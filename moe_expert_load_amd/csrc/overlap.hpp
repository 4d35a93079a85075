// Host-side check of tensor ranges.
#pragma once

#include <stdint.h>

namespace moonep {

// Whether two byte ranges share memory.
inline bool overlap(const void* a, int64_t na, const void* b, int64_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && x < y + (uintptr_t)nb && y < x + (uintptr_t)na;
}

}  // namespace moonep
