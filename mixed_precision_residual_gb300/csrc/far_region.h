// Strided regions of memory and the overlap tests behind the aliasing rules (host only).
#pragma once

#include <stdint.h>

namespace far {

// A strided tensor in memory: `rows` rows of `width` bytes, `stride` bytes apart.
struct Region {
  uint64_t base;
  int64_t rows, width, stride;
};

inline Region region(const void* p, int64_t rows, int64_t width, int64_t stride) {
  return Region{(uint64_t)(uintptr_t)p, rows, width, stride};
}

inline int64_t floor_div(int64_t a, int64_t b) {  // b > 0
  return a >= 0 ? a / b : -((-a + b - 1) / b);
}

// Do any bytes of A and B coincide?  Exact for equal strides (rows of two column
// slices of one matrix interleave without touching); otherwise any overlap of the
// spanned byte ranges counts.
inline bool regions_overlap(const Region& A, const Region& B) {
  if (A.rows == 0 || B.rows == 0 || A.width == 0 || B.width == 0) return false;
  const uint64_t a_end = A.base + (uint64_t)((A.rows - 1) * A.stride + A.width);
  const uint64_t b_end = B.base + (uint64_t)((B.rows - 1) * B.stride + B.width);
  if (!(A.base < b_end && B.base < a_end)) return false;
  if (A.stride != B.stride || A.rows == 1 || B.rows == 1) return true;
  // row i of A and row j of B meet iff -B.width < d + (j - i) * s < A.width, d = B.base - A.base
  const int64_t s = A.stride;
  const int64_t d = (int64_t)(B.base - A.base);
  const int64_t kmin = floor_div(-B.width - d, s) + 1;
  const int64_t kmax = -floor_div(-(A.width - d), s) - 1;  // ceil((A.width - d) / s) - 1
  const int64_t lo = kmin > -(A.rows - 1) ? kmin : -(A.rows - 1);  // j - i, 0 <= i < A.rows, 0 <= j < B.rows
  const int64_t hi = kmax < (B.rows - 1) ? kmax : (B.rows - 1);
  return lo <= hi;
}

inline bool same_region(const Region& A, const Region& B) {
  return A.base == B.base && A.rows == B.rows && A.width == B.width && A.stride == B.stride;
}

// an output may be exactly an input region (in place); no other byte may be shared
inline bool bad_overlap(const Region& out, const Region& in) { return regions_overlap(out, in) && !same_region(out, in); }

}  // namespace far
