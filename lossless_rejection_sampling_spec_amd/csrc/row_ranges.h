// row_ranges.h -- whether two arrays of strided rows have memory in common (host code).
#pragma once

#include <stdint.h>

namespace svk {

// Arrays of `rows` rows of `width` bytes, ld_a and ld_b bytes apart (at least `width`).  Columns
// of one wider array share its range of addresses and may still have no byte in common.
inline bool rows_overlap(const void* a, int64_t ld_a, const void* b, int64_t ld_b, int64_t rows,
                         int64_t width) {
  typedef __int128 wide;                      // (rows * ld of any call fits)
  const wide pa = (uintptr_t)a, pb = (uintptr_t)b;
  if (pa + (rows - 1) * (wide)ld_a + width <= pb || pb + (rows - 1) * (wide)ld_b + width <= pa)
    return false;
  if (ld_a == ld_b) {                         // the two row distances around the arrays' own
    const wide gap = pb > pa ? pb - pa : pa - pb, whole = gap / ld_a;
    return gap - whole * ld_a < width || (whole + 1 < rows && (whole + 1) * ld_a - gap < width);
  }
  wide x = pa, y = pb;                        // rows in the order of their addresses
  for (int64_t i = 0, j = 0; i < rows && j < rows;) {
    if (x + width <= y) ++i, x += ld_a;
    else if (y + width <= x) ++j, y += ld_b;
    else return true;
  }
  return false;
}

}  // namespace svk
