// fp4_ranges.hpp -- the index arithmetic of the MXFP4 kernels where it meets the ends of its types and
// arrays, in plain constexpr C++ (host and device), so that the host can check it at sizes that no test
// would allocate.
#pragma once
#include <stdint.h>

namespace mxq {

// Columns 0 .. n-1 (1 <= n < 2^31) are stored in groups of four: their number, and whether the group
// that begins at `col` (a multiple of 4 below n) is whole.  No sum here passes n, which may be 2^31 - 1.
constexpr int column_groups(int n) { return (n - 1) / 4 + 1; }
constexpr bool whole_group(int col, int n) { return n - col >= 4; }

// Bytes from the first of `rows` rows of scales to the last one's end: its nb bytes, or, where rows are read
// by 4-byte words, the word that holds the last of them.  What lies behind may be another's, or no memory.
constexpr uint32_t scale_bytes(int64_t rows, int64_t ld, int nb, bool words) {
  return (uint32_t)((rows - 1) * ld + (words ? (nb + 3) & ~3 : nb));
}

// The grid of n workgroups (n < 2^31).  A launch takes less than 2^32 threads along x, 2^23 workgroups of
// 512, so more than 2^22 workgroups continue along y; those that fill up the last row, numbers from n on,
// have nothing to do (a kernel asks only where y > 0: the question waits for its arguments).  2^22 is a multiple of the XCDs, so the order in which they are dealt goes on.
constexpr int kGridX = 1 << 22;
struct Grid {
  uint32_t x, y;
};
constexpr Grid grid_of(int64_t n) {
  return n <= kGridX ? Grid{(uint32_t)n, 1} : Grid{(uint32_t)kGridX, (uint32_t)((n + kGridX - 1) / kGridX)};
}
constexpr int workgroup_at(uint32_t x, uint32_t y) { return (int)(x + y * kGridX); }

}  // namespace mxq
