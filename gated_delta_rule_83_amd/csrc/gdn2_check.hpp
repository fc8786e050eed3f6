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

// Whether p is aligned to its elements of `bytes` bytes.
inline bool aligned_to(const void *p, size_t bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) == 0; }

// Outputs against inputs and against each other; out[i] may be in[same[i]]
// exactly (-1: none).
inline bool outputs_overlap(const Range *in, int ni, const Range *out, int no, const int *same) {
  for (int i = 0; i < no; ++i) {
    for (int j = 0; j < ni; ++j) {
      if (same && same[i] == j && out[i].lo == in[j].lo) continue;
      if (overlaps(out[i], in[j])) return true;
    }
    for (int j = i + 1; j < no; ++j)
      if (overlaps(out[i], out[j])) return true;
  }
  return false;
}

inline size_t ceil_div(size_t x, size_t y) { return (x + y - 1) / y; }

constexpr size_t kMaxGroups = (1u << 24) - 1;  // workgroups of 256 threads of one launch

}  // namespace gdn2
