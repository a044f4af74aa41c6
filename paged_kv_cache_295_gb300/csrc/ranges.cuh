// Ranges of bytes that a call's arguments take.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace pkv {

// Whether two ranges have a byte in common.
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a && b && na && nb && x < y + nb && y < x + na;
}

}  // namespace pkv
