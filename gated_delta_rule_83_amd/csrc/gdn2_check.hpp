// gdn2_check.hpp -- argument checks shared by the C ABI's entry points: byte
// ranges of the caller's buffers, their overlaps and their alignment.
#pragma once

#include <stddef.h>
#include <stdint.h>

namespace gdn2 {

struct Range {
  uintptr_t lo, hi;  // [lo, hi)
};

inline Range range_of(const void *p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return Range{lo, lo + bytes};
}

inline bool overlaps(Range x, Range y) {
  return x.lo != x.hi && y.lo != y.hi && x.lo < y.hi && y.lo < x.hi;
}

inline bool aligned16(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
// One fp32 per token and value head (beta, alpha and their gradients) is read
// and written as single floats: 4-byte alignment, so that a view starting at
// any token of a [T, H_v] tensor is accepted.
inline bool aligned4(const void *p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

}  // namespace gdn2
