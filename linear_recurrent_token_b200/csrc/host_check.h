// Pointer checks shared by the C entry points.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace mlstm {

inline bool misaligned(const void* p) { return ((uintptr_t)p & 15) != 0; }

struct Range {
  const void* p;
  size_t n;
};
inline bool overlaps(Range a, Range b) {
  if (!a.p || !b.p || a.n == 0 || b.n == 0) return false;
  const uintptr_t a0 = (uintptr_t)a.p, b0 = (uintptr_t)b.p;
  return a0 < b0 + b.n && b0 < a0 + a.n;
}

}  // namespace mlstm
