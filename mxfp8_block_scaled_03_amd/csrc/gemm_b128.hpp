// gemm_b128.hpp -- what the kernels of the product in blocks of 128 share (gemm_b128_tile.hip: 256 x 256
// tiles; gemm_b128_mid.hip: 128 x 128 and 64 x 64; gemm_b128_rows.hip: small tiles whose waves split K): the
// problem, the tile that a workgroup takes, the matrix instructions of one block, the epilogue's arithmetic.
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
typedef int v4i_any __attribute__((ext_vector_type(4), aligned(1)));

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
    const Group g = find_group_by(a.offsets, a.experts, a.M, TM, tiles_n, wg,
                                  [](int t, int total) { return XCD ? xcd_order(t, total) : t; });
    if (g.e < 0) return t;
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
    // experts in turn, each in XCD order: their lengths differ, and an XCD that had one expert's tiles to itself would
    // finish early or late (8192 rows over 4 experts, 4096 x 2048 exact: 262 us instead of 197)
    const int e = wg / each;
    tile_at(xcd_order(wg % each, each), tiles_m, tiles_n, tm, tn);
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
__device__ __forceinline__ float finish(float acc, float alpha, float bias, int act) {
  const float v = __builtin_fmaf(alpha, acc, bias);
  return act ? silu(v) : v;
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// 4 bytes per lane from buffer offset voff into LDS at lds + 4 * lane.
__device__ __forceinline__ void dma4(uint32_t lds, uint32_t voff, v4i rsrc) {
  asm volatile("s_mov_b32 m0, %0\n\tbuffer_load_dword %1, %2, 0 offen lds"
               :
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
#pragma clang diagnostic pop

// Four sums of a wave that have to be there at this point: results of vector instructions, never of matrix ones.
template <int N>
__device__ __forceinline__ void pin(v4f (&a)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) asm volatile("" : "+v"(a[j]));
}

// The epilogue of a wave that holds 16 FM x 16 FN outputs: lane (i, g) has Y[row0 + 16 f + i][col0 + 16 j + 4 g + r]
// of the tile in acc[f][j][r].  act(alpha v + bias), then rows of 16 FN values through REGION bytes of LDS of the
// wave's own, 16-byte piece c of row r at c ^ (r & 7), and out in 16-byte pieces, value by value in the last
// columns.  PAST: past the caches.
template <int E, bool PAST, int FM, int FN, int REGION>
__device__ __forceinline__ void store_rows(const GemmB128& a, const B128Tile& t, const v4f (&acc)[FM][FN], int wid, int lane,
                                           int row0, int col0) {
  constexpr int RB = 16 * FN * E, CPR = RB / 16, RP = REGION / RB < 16 * FM ? REGION / RB : 16 * FM, FPP = RP / 16;
  constexpr int XOR = (CPR < 8 ? CPR : 8) - 1;
  static_assert(RP % 16 == 0 && FM % FPP == 0 && 1024 % RB == 0, "rows of a pass");
  const int i = lane & 15, g = lane >> 4;
  const uint32_t base = (uint32_t)wid * REGION;
#pragma unroll
  for (int pass = 0; pass < FM / FPP; ++pass) {
#pragma unroll
    for (int j = 0; j < FN; ++j)
#pragma unroll
      for (int fl = 0; fl < FPP; ++fl) {
        const int f = pass * FPP + fl, row = 16 * fl + i;
        const uint32_t byte = (uint32_t)((16 * j + 4 * g) * E);
        const uint32_t at = base + (uint32_t)row * RB + (((byte >> 4) ^ (uint32_t)(row & XOR)) << 4) + (byte & 15);
        if (E == 2) {
          const v2u p = {pack_bf16(acc[f][j][0], acc[f][j][1]), pack_bf16(acc[f][j][2], acc[f][j][3])};
          *reinterpret_cast<v2u*>(smem + at) = p;
        } else {
          *reinterpret_cast<v4f*>(smem + at) = acc[f][j];
        }
      }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
    constexpr int RPI = 1024 / RB;
    const int c = lane % CPR, left = t.n - col0 - c * (16 / E);   // columns from this piece on
#pragma unroll 4
    for (int it = 0; it < RP / RPI; ++it) {
      const int row = it * RPI + lane / CPR, m = row0 + pass * RP + row;
      const v4i v = lds16(base + (uint32_t)row * RB + (uint32_t)((c ^ (row & XOR)) << 4), 0);
      if (m >= t.m) continue;
      uint8_t* dst = reinterpret_cast<uint8_t*>(a.y) + (t.y + (int64_t)m * a.ld_y + col0) * E + 16 * c;
      if (left >= 16 / E) {
        v4i_any* out = reinterpret_cast<v4i_any*>(dst);     // one store, whatever y's alignment
        if (PAST)
          __builtin_nontemporal_store((v4i_any)v, out);
        else
          *out = v;
      } else {
#pragma unroll
        for (int q = 0; q < 16 / E; ++q)
          if (q < left) {
            if (E == 2)
              reinterpret_cast<uint16_t*>(dst)[q] = (uint16_t)((uint32_t)v[q >> 1] >> (16 * (q & 1)));
            else
              reinterpret_cast<uint32_t*>(dst)[q] = (uint32_t)v[q];
          }
      }
    }
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront", "local");
    __builtin_amdgcn_wave_barrier();
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront", "local");
  }
}

template <int FM, int FN, int REGION>
__device__ __forceinline__ void epilogue(const GemmB128& a, const B128Tile& t, v4f (&acc)[FM][FN], int wid, int lane, int row0,
                                         int col0) {
  const bool has_bias = a.bias != nullptr;
  // (from the tile's first column on: offsets from the first of all pass 2^31 bytes in column 2^29)
  const __amdgpu_buffer_rsrc_t brs = bias_rsrc(has_bias ? a.bias + t.n0 : nullptr, t.n);
#pragma unroll
  for (int j = 0; j < FN; ++j) {
    const int col = col0 + 16 * j + 4 * (lane >> 4);
    const v4f bq = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(brs, 4 * col, 0, 0));
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float bv = has_bias && col + r < t.n ? bq[r] : -0.0f;
#pragma unroll
      for (int f = 0; f < FM; ++f) acc[f][j][r] = finish(acc[f][j][r], a.alpha, bv, a.act);
    }
  }
  if (a.past_caches) {
    if (a.y_bf16)
      store_rows<2, true, FM, FN, REGION>(a, t, acc, wid, lane, row0, col0);
    else
      store_rows<4, true, FM, FN, REGION>(a, t, acc, wid, lane, row0, col0);
  } else {
    if (a.y_bf16)
      store_rows<2, false, FM, FN, REGION>(a, t, acc, wid, lane, row0, col0);
    else
      store_rows<4, false, FM, FN, REGION>(a, t, acc, wid, lane, row0, col0);
  }
}

}  // namespace
}  // namespace mxq
