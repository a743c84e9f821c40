// b128.hpp -- FP8 codes in blocks of 128 with FP32 scales: what the quantizer (quantize_b128.hip) and the
// products (gemm_b128*.hip) share.
//
// A block is 128 consecutive values of a line along the contraction axis, or a tile of 128 lines by 128
// values; x ~ s * code with one FP32 scale s.  Code lines hold whole blocks (128 bytes each, zero past the
// last value), so the products need no masks along K.  The scales of one block of many lines lie side by
// side, [block][line]: a product's tile reads its 256 lines' scales of a step as one run, and a quantizer's
// tile writes them as one.
//
// Experts: lines sorted by expert, expert e's being offsets[e] .. offsets[e+1] - 1, offsets on the device.
// Where K runs along those lines (the weight gradient), each expert's lines begin a block of their own.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

namespace mxq {

constexpr int kB = 128;   // values in a block

// The most blocks (or tiles of `size` lines) that `rows` lines can take when each of `groups` experts' lines
// begin a new one: the sum of ceil(n_e / size) is at most (rows + groups (size - 1)) / size.
constexpr int64_t grouped_tiles(int64_t rows, int64_t groups, int64_t size) {
  return (rows + groups * (size - 1)) / size;
}

#ifdef __HIPCC__
struct Group {
  int e;        // the expert, -1 where no expert has the tile
  int row0;     // the tile's first line
  int rows;     // its expert's lines from there on
  int tile;     // the tile's number among its expert's
  int tiles;    // how many its expert has
  int total;    // tiles of all experts
};

// Tile number `t` (of `size` lines each, every expert's first line beginning a tile) -> its expert and lines.
// Every wave searches for itself, 64 experts at a time: a tile count per lane, a scan over the lanes, the
// first lane whose sum passes t.  Offsets are taken into 0 .. rows and in order, so that wrong ones cannot
// lead outside the lines.  `scale` tiles count for each tile of lines (the tiles along the other axis), and
// Group::tile counts those.
__device__ __forceinline__ Group find_group(const int* __restrict__ offsets, int experts, int rows, int size, int scale,
                                            int t) {
  const int lane = threadIdx.x & 63;
  Group g{-1, 0, 0, 0, 0, 0};
  int before = 0;
  for (int e0 = 0; e0 < experts; e0 += 64) {
    const int e = e0 + lane;
    int lo = 0, n = 0;
    if (e < experts) {
      lo = min(max(offsets[e], 0), rows);
      n = max(min(offsets[e + 1], rows), lo) - lo;
    }
    const int mine = ((n + size - 1) / size) * scale;
    int sum = mine;
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) {
      const int o = __shfl_up(sum, d, 64);
      sum += lane >= d ? o : 0;
    }
    const uint64_t past = __ballot(before + sum > t);
    if (g.e < 0 && past) {
      const int l = __builtin_ctzll(past);
      g.e = e0 + l;
      g.row0 = __builtin_amdgcn_readlane(lo, l);
      g.rows = __builtin_amdgcn_readlane(n, l);
      g.tiles = __builtin_amdgcn_readlane(mine, l);
      g.tile = t - (before + __builtin_amdgcn_readlane(sum, l) - g.tiles);
    }
    before += __builtin_amdgcn_readlane(sum, 63);
  }
  g.total = before;
  return g;
}

// The same for tile order(t, tiles of all experts), -1 where there are no more than t tiles.
template <typename Order>
__device__ __forceinline__ Group find_group_by(const int* __restrict__ offsets, int experts, int rows, int size, int scale,
                                               int t, Order order) {
  if (experts > 64) {
    const Group g = find_group(offsets, experts, rows, size, scale, 0x7FFFFFFF);
    return t >= g.total ? g : find_group(offsets, experts, rows, size, scale, order(t, g.total));
  }
  // one search, since the sums are there when the number of tiles is (8192 rows of 32 experts of 4096 x 2048, quantized
  // too, 132 us by two, 129 so)
  const int lane = threadIdx.x & 63;
  int lo = 0, n = 0;
  if (lane < experts) {
    lo = min(max(offsets[lane], 0), rows);
    n = max(min(offsets[lane + 1], rows), lo) - lo;
  }
  const int mine = ((n + size - 1) / size) * scale;
  int sum = mine;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int o = __shfl_up(sum, d, 64);
    sum += lane >= d ? o : 0;
  }
  Group g{-1, 0, 0, 0, 0, 0};
  g.total = __builtin_amdgcn_readlane(sum, 63);
  if (t >= g.total) return g;
  const int at = order(t, g.total), l = __builtin_ctzll(__ballot(sum > at));
  g.e = l;
  g.row0 = __builtin_amdgcn_readlane(lo, l);
  g.rows = __builtin_amdgcn_readlane(n, l);
  g.tiles = __builtin_amdgcn_readlane(mine, l);
  g.tile = at - (__builtin_amdgcn_readlane(sum, l) - g.tiles);
  return g;
}
#endif

}  // namespace mxq
