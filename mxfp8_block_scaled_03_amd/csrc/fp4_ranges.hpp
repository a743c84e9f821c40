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

}  // namespace mxq
