// api_check.hpp -- pointer checks shared by the C-ABI sources.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gdr {
namespace check {

inline bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) % n) == 0; }

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void* p, size_t bytes) {
  uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + bytes};
}

inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi && a.lo != a.hi && b.lo != b.hi; }

inline bool overlaps_any(Range a, const Range* others, int n) {
  for (int i = 0; i < n; ++i)
    if (overlap(a, others[i])) return true;
  return false;
}

}  // namespace check
}  // namespace gdr
