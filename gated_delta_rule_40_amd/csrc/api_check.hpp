// api_check.hpp -- size and pointer checks shared by the C-ABI sources.
#pragma once

#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

#include <hip/hip_runtime_api.h>

#include "gdr.h"

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

inline Range range_or_none(const void* p, size_t bytes) {
  return p ? range_of(p, bytes) : Range{0, 0};
}

// Writes must keep clear of every read and of each other.
template <int NW, int NR>
bool clash(const Range (&writes)[NW], const Range (&reads)[NR]) {
  for (int i = 0; i < NW; ++i) {
    if (overlaps_any(writes[i], reads, NR)) return true;
    for (int j = i + 1; j < NW; ++j)
      if (overlap(writes[i], writes[j])) return true;
  }
  return false;
}

// Bytes from the first to behind the last element of rows `stride` apart.
inline size_t rows_extent(size_t rows, int64_t stride, size_t width, size_t es) {
  return rows ? ((rows - 1) * static_cast<size_t>(stride) + width) * es : 0;
}

inline bool known_io(gdr_dtype io) { return io == GDR_F32 || io == GDR_BF16; }
inline size_t size_of(gdr_dtype io) { return io == GDR_BF16 ? 2 : 4; }

inline int result(hipError_t e) { return e == hipSuccess ? GDR_OK : GDR_E_HIP; }

// Whether a product of non-negative factors stays within `limit`.
inline bool within(long long limit, std::initializer_list<long long> factors) {
  long long p = 1;
  for (long long f : factors) {
    if (f != 0 && p > limit / f) return false;
    p *= f;
  }
  return true;
}

}  // namespace check
}  // namespace gdr
