// gemm_b128.hpp -- what the two kernels of the product in blocks of 128 share (gemm_b128_tile.hip: 256 x 256
// tiles; gemm_b128_rows.hip: small tiles whose waves split K): the problem, the tile that a workgroup takes,
// the matrix instructions of one block, the epilogue's arithmetic.
//
// Y[m][n] = act(alpha sum_b sx[m][b] sw[n][b] (sum_{k in b} qx[m][k] qw[n][k]) + bias[n]).  The inner sum is a
// matrix product of codes from zero, the outer one FP32 fused multiply-adds on the vector unit, one for each
// output and block.  The matrix instruction takes W as its A operand and X as its B operand, so that a lane
// holds four consecutive n of one m: where W's scales are those of tiles, the factor sx sw is one number for
// all that a lane has of a 16 x 16 tile.
#pragma once
#include "b128.hpp"
#include "fp4_ranges.hpp"
#include "gemm_common.hpp"

namespace mxq {

namespace {
typedef float v4f __attribute__((ext_vector_type(4)));
typedef uint32_t v2u __attribute__((ext_vector_type(2)));

// What a workgroup multiplies: lines of X and W from the tile's first on, `nb` blocks of K, and where Y goes.
struct B128Tile {
  bool any;
  const uint8_t *x, *w;
  const float *xs, *ws;     // ws: the first line's (tile's) scale of the first block
  int m, n;                 // lines left of X and W from here on
  int nb;
  int64_t y;                // element offset of the tile in y
  int n0;                   // first column, for the bias
};

// Tile `wg` of TM x TN outputs.  Plain: tiles of one matrix in XCD order.  Rows of experts: each expert's
// tiles in turn, W and its scales the expert's.  Blocks of experts (the weight gradient): every expert has
// the whole matrix of tiles, its blocks of K only.
template <int TM, int TN, bool WLINE, bool XCD = true>
__device__ __forceinline__ B128Tile b128_tile(const GemmB128& a, int wg) {
  B128Tile t{};
  int tm, tn;
  const int tiles_n = (a.N + TN - 1) / TN;
  int64_t wrow = 0;
  t.nb = a.nb;
  if (a.mode == kB128Plain) {
    const int tiles_m = (a.M + TM - 1) / TM;
    if (wg >= tiles_m * tiles_n) return t;
    tile_of(wg, tiles_m, tiles_n, tm, tn);
    t.m = a.M - tm * TM;
    t.x = a.x + (int64_t)tm * TM * a.ld_x;
    t.xs = a.xs + tm * TM;
    t.w = a.w;
    t.ws = a.ws;
    t.y = (int64_t)tm * TM * a.ld_y;
  } else if (a.mode == kB128Rows) {
    // the grid is an upper bound: the tiles that there are come first, in XCD order where tiles share operands
    Group g = find_group(a.offsets, a.experts, a.M, TM, tiles_n, XCD ? 0x7FFFFFFF : wg);
    if (wg >= g.total) return t;
    if (XCD) g = find_group(a.offsets, a.experts, a.M, TM, tiles_n, xcd_order(wg, g.total));
    tile_at(g.tile, g.tiles / tiles_n, tiles_n, tm, tn);
    const int64_t row = g.row0 + (int64_t)tm * TM;
    t.m = g.rows - tm * TM;
    t.x = a.x + row * a.ld_x;
    t.xs = a.xs + row;
    t.w = a.w + g.e * a.st_w;
    t.ws = a.ws + g.e * a.st_ws;
    t.y = row * a.ld_y;
  } else {
    const int tiles_m = (a.M + TM - 1) / TM, each = tiles_m * tiles_n;
    if (wg >= each * a.experts) return t;
    const int at = xcd_order(wg, each * a.experts), e = at / each;
    tile_at(at % each, tiles_m, tiles_n, tm, tn);
    // the expert's first block: the blocks of those before it
    int first = 0, lane = threadIdx.x & 63;
    for (int e0 = 0; e0 <= e; e0 += 64) {
      int n = 0;
      if (e0 + lane <= e) {
        const int lo = min(max(a.offsets[e0 + lane], 0), a.rows);
        n = (max(min(a.offsets[e0 + lane + 1], a.rows), lo) - lo + kB - 1) / kB;
      }
      if (e0 + 64 > e) t.nb = __builtin_amdgcn_readlane(n, e - e0);
      int sum = n;
#pragma unroll
      for (int d = 32; d > 0; d >>= 1) sum += __shfl_xor(sum, d, 64);
      first += __builtin_amdgcn_readfirstlane(sum);
    }
    first -= t.nb;
    first = min(first, a.nb);            // (wrong offsets must not lead outside the lines)
    t.nb = min(t.nb, a.nb - first);
    t.m = a.M - tm * TM;
    t.x = a.x + (int64_t)tm * TM * a.ld_x + (int64_t)first * kB;
    t.xs = a.xs + first * a.ld_xs + tm * TM;
    t.w = a.w + (int64_t)first * kB;
    t.ws = a.ws + first * a.ws_k;
    t.y = e * a.st_y + (int64_t)tm * TM * a.ld_y;
  }
  t.any = true;
  t.n0 = tn * TN;
  t.n = a.N - t.n0;
  wrow = t.n0;
  t.w += wrow * a.ld_w;
  t.ws += WLINE ? wrow : (wrow / kB) * a.ws_n;
  t.y += t.n0;
  return t;
}

// The sum over one block of 16 lines of W (its 32 codes a lane, in two 16-byte halves) and 16 of X.
// FP8 matrix cores: v_mfma_f32_16x16x128_f8f6f4, one for the block.  Exact: the codes as bf16, four times
// v_mfma_f32_16x16x32_bf16; which k a lane holds does not matter as long as it is the same for both operands.
template <int FX, int FW>
__device__ __forceinline__ v4f block_fp8(v8i w, v8i x) {
  const v4f zero = {0.0f, 0.0f, 0.0f, 0.0f};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x, zero, FW, FX, 0, 0, 0, 0);
}

struct Wide {
  v8bf p[4];
};
template <int F>
__device__ __forceinline__ Wide widen(v8i c) {
  Wide r;
#pragma unroll
  for (int q = 0; q < 4; ++q) r.p[q] = codes_to_bf16<F>((uint32_t)c[2 * q], (uint32_t)c[2 * q + 1], 1.0f);
  return r;
}
__device__ __forceinline__ v4f block_exact(const Wide& w, const Wide& x) {
  v4f t = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int q = 0; q < 4; ++q) t = __builtin_amdgcn_mfma_f32_16x16x32_bf16(w.p[q], x.p[q], t, 0, 0, 0);
  return t;
}

__device__ __forceinline__ float finish(float acc, float alpha, float bias, int act) {
  const float v = __builtin_fmaf(alpha, acc, bias);
  return act ? silu(v) : v;
}

}  // namespace
}  // namespace mxq
