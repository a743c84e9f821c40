// quantize_b128.hip -- FP8 codes and FP32 scales in blocks of 128 (mxq_quantize_b128).
//
// Mathematics: a = max |x| over the block, s = fl(a / fmax), r = fl(fmax / a), code = RNE8(fl(x r)); a zero
// block has s = r = 1, and a block below 2^-100 takes a = 2^-100, so that s and r stay normal numbers.  fl is
// FP32's nearest even.  |x| r <= fmax (1 + 2^-23), far below the midpoint past fmax, so no code saturates.
// Under the ceil rule s is the power of two that the MXFP8 quantizer would take, r its exact inverse.  A NaN
// or an infinity in a block makes s NaN and every code of the block 0x7F.
//
// Bound by HBM: 2 or 4 bytes read and 1 or 2 written for each value.  One workgroup of 256 threads holds a
// 128 x 128 tile in registers, so that both orientations (and the tile's own maximum) come from one read:
// thread (rg, c) has rows 8 rg .. 8 rg + 7 of the eight columns 8 c .. 8 c + 7.  A row's 16 threads lie in
// one 16-lane row of a wave, so its maximum takes four lane steps; a column's is taken over the thread's
// eight rows, two lane steps and four waves in LDS.  The eight rows of a column are eight consecutive bytes
// of the transposed codes: they go through LDS as one 8-byte word and leave as 16-byte pieces, eight lanes to
// a 128-byte line.
#include <type_traits>

#include "b128.hpp"
#include "codec.hpp"
#include "internal.hpp"
#include "mxblock.hpp"

namespace mxq {
namespace {

struct QuantArgs {
  const void* src;
  int64_t rows, cols, ld;
  uint8_t* rc;
  int64_t ld_rc;
  float* rs;
  int64_t ld_rs;
  uint8_t* cc;
  int64_t ld_cc;
  float* cs;
  int64_t ld_cs;
  const int* offsets;
  int experts, rule, vec, blocks_c;   // blocks_c: blocks that a line of cc and cs has room for
  int tiles_r, tiles_c;
};

// Scale and factor of a block from the bits of its maximum.
template <int F>
__device__ __forceinline__ void scale_of(uint32_t abits, int rule, float& s, float& r) {
  constexpr float fmax = F == kE4M3 ? 448.0f : 57344.0f;
  s = r = 1.0f;
  if (abits == 0) return;
  if (abits >= 0x7F800000u) {
    s = __uint_as_float(0x7FC00000u);
    return;
  }
  const float a = fmaxf(__uint_as_float(abits), 0x1p-100f);
  if (rule == 0) {
    s = a / fmax;
    r = fmax / a;
  } else {
    const uint32_t u = __float_as_uint(a);
    const uint32_t e = (u >> 23) - Fp8<F>::emax + ((u & 0x7FFFFFu) > 0x600000u ? 1u : 0u);
    s = __uint_as_float(e << 23);
    r = __uint_as_float((254u - e) << 23);
  }
}

// The largest of the 16 lanes of a row of lanes.
__device__ __forceinline__ uint32_t row16_max(uint32_t v) {
  uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x128, 0xF, 0xF, false);   // row_ror:8
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x124, 0xF, 0xF, false);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x122, 0xF, 0xF, false);
  v = v > o ? v : o;
  o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, 0x121, 0xF, 0xF, false);
  return v > o ? v : o;
}

// Eight values under eight factors (or one): two dwords of codes.
template <int F>
__device__ __forceinline__ void encode8(const float v[8], const float r[8], const bool bad[8], uint32_t d[2]) {
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = __float_as_uint(v[4 * h + e] * r[4 * h + e]);
    uint32_t w = mxblock::cvt2_f32<F>(0u, p[0], p[1], 1.0f, false);
    w = mxblock::cvt2_f32<F>(w, p[2], p[3], 1.0f, true);
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (bad[4 * h + e]) w = (w & ~(0xFFu << (8 * e))) | (0x7Fu << (8 * e));
    d[h] = w;
  }
}

// Q rows a thread (8, or 1 where rows alone are wanted and few tiles of 128 rows would leave the card empty).
template <int BF16, int F, bool ROW, bool COL, bool TILE, int Q>
__global__ __launch_bounds__(256) void k_quant_b128(const QuantArgs a) {
  constexpr int kRows = 16 * Q;
  __shared__ uint32_t s_max[4][COL ? kB : 1];
  __shared__ __attribute__((aligned(16))) uint8_t s_codes[COL ? kB * kB : 16];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = tid & 15, rg = tid >> 4;
  const int bc = blockIdx.x % a.tiles_c, tr = blockIdx.x / a.tiles_c;
  int64_t row0 = (int64_t)tr * kRows;
  int rows = (int)min((int64_t)kRows, a.rows - row0), out_block = tr;
  if (COL && a.offsets) {
    const Group g = find_group(a.offsets, a.experts, (int)a.rows, kB, 1, tr);
    if (g.e < 0 || tr >= a.blocks_c) return;
    row0 = g.row0 + kB * g.tile;
    rows = min(kB, g.rows - kB * g.tile);
  }
  const int64_t col = (int64_t)bc * kB + 8 * c;
  const int cols = (int)min((int64_t)8, a.cols - col);   // of this thread's eight, 0 or less past the end
  float v[Q][8];
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    const int r = Q * rg + q;
    const int64_t at = (row0 + r) * a.ld + col;
    if (r < rows && cols == 8 && a.vec) {
      if (BF16) {
        const uint4 u = *reinterpret_cast<const uint4*>(reinterpret_cast<const uint16_t*>(a.src) + at);
        const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
        for (int e = 0; e < 8; ++e) v[q][e] = __uint_as_float(e & 1 ? w[e >> 1] & 0xFFFF0000u : w[e >> 1] << 16);
      } else {
        const float4* p = reinterpret_cast<const float4*>(reinterpret_cast<const float*>(a.src) + at);
        const float4 lo = p[0], hi = p[1];
        v[q][0] = lo.x, v[q][1] = lo.y, v[q][2] = lo.z, v[q][3] = lo.w;
        v[q][4] = hi.x, v[q][5] = hi.y, v[q][6] = hi.z, v[q][7] = hi.w;
      }
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        v[q][e] = 0.0f;
        if (r < rows && e < cols)
          v[q][e] = BF16 ? __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.src)[at + e] << 16)
                         : reinterpret_cast<const float*>(a.src)[at + e];
      }
    }
  }
  uint32_t rmax[Q], cmax[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) cmax[e] = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    rmax[q] = 0;
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t u = __float_as_uint(v[q][e]) & 0x7FFFFFFFu;
      rmax[q] = max(rmax[q], u);
      if (COL) cmax[e] = max(cmax[e], u);
    }
  }
  float tile_s = 1.0f, tile_r = 1.0f;
  bool tile_bad = false;
  if (TILE) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) m = max(m, rmax[q]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    if (lane == 0) s_max[wave][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < 4; ++w) m = max(m, s_max[w][0]);
    scale_of<F>(m, a.rule, tile_s, tile_r);
    tile_bad = m >= 0x7F800000u;
    if (tid == 0) a.rs[(int64_t)tr * a.ld_rs + bc] = tile_s;
  }
  if (ROW) {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = Q * rg + q;
      float s = tile_s, f = tile_r;
      bool b = tile_bad;
      if (!TILE) {
        const uint32_t m = row16_max(rmax[q]);
        scale_of<F>(m, a.rule, s, f);
        b = m >= 0x7F800000u;
        if (c == 0 && r < rows) a.rs[(int64_t)bc * a.ld_rs + row0 + r] = s;
      }
      float fs[8];
      bool bs[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) fs[e] = f, bs[e] = b && e < cols;
      uint32_t d[2];
      encode8<F>(v[q], fs, bs, d);
      if (r < rows)
        *reinterpret_cast<uint2*>(a.rc + (row0 + r) * a.ld_rc + (int64_t)bc * kB + 8 * c) = make_uint2(d[0], d[1]);
    }
  }
  if (COL) {
    float f[8];
    bool b[8];
    if (TILE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = tile_r, b[e] = tile_bad;
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        cmax[e] = max(cmax[e], (uint32_t)__shfl_xor((int)cmax[e], 16, 64));
        cmax[e] = max(cmax[e], (uint32_t)__shfl_xor((int)cmax[e], 32, 64));
      }
      if (lane < 16) {
#pragma unroll
        for (int e = 0; e < 8; ++e) s_max[wave][8 * c + e] = cmax[e];
      }
      __syncthreads();
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        uint32_t m = 0;
#pragma unroll
        for (int w = 0; w < 4; ++w) m = max(m, s_max[w][8 * c + e]);
        float s;
        scale_of<F>(m, a.rule, s, f[e]);
        b[e] = m >= 0x7F800000u;
        if (rg == 0 && e < cols) a.cs[(int64_t)out_block * a.ld_cs + col + e] = s;
      }
    }
    // the eight codes of column 8 c + j, rows 8 rg .. 8 rg + 7, as an 8-byte word.  LDS row 8 c + (j ^ (c & 1))
    // of 16 words, word rg ^ (c & 14): the 32 lanes that write together touch every bank once.
    uint32_t w[8][2];
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x[8], fs[8];
      bool bs[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = v[q & (Q - 1)][j], fs[q] = f[j], bs[q] = b[j] && 8 * rg + q < rows;
      encode8<F>(x, fs, bs, w[j]);
    }
#pragma unroll
    for (int j = 0; j < 8; ++j)
      *reinterpret_cast<uint2*>(s_codes + (8 * c + (j ^ (c & 1))) * kB + 8 * (rg ^ (c & 14))) = make_uint2(w[j][0], w[j][1]);
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int k = 32 * it + (tid >> 3), p = tid & 7, kc = k >> 3;   // column k, rows 16 p .. 16 p + 15
      const uint4 u = *reinterpret_cast<const uint4*>(s_codes + (8 * kc + ((k & 7) ^ (kc & 1))) * kB + 8 * ((2 * p) ^ (kc & 14)));
      if ((int64_t)bc * kB + k < a.cols)
        *reinterpret_cast<uint4*>(a.cc + ((int64_t)bc * kB + k) * a.ld_cc + (int64_t)out_block * kB + 16 * p) = u;
    }
  }
}

template <int BF16, int F>
hipError_t launch_f(const QuantArgs& args, bool row, bool col, bool tile, hipStream_t stream) {
  QuantArgs a = args;
  a.tiles_c = (int)((a.cols + kB - 1) / kB);
  const int64_t tiles = a.offsets ? grouped_tiles(a.rows, a.experts, kB) : (a.rows + kB - 1) / kB;
  // rows alone: tiles of 16 rows where tiles of 128 would be fewer than two for each CU
  const bool thin = !col && !tile && tiles * a.tiles_c < 2 * (int64_t)device_cu_count();
  const int64_t tr = thin ? (a.rows + 15) / 16 : tiles;
  if (tr * a.tiles_c > 0x7FFFFF) return hipErrorInvalidValue;
  a.tiles_r = (int)tr;
  const dim3 grid((unsigned)(tr * a.tiles_c)), block(256);
  if (tile && col)
    hipLaunchKernelGGL((k_quant_b128<BF16, F, true, true, true, 8>), grid, block, 0, stream, a);
  else if (tile)
    hipLaunchKernelGGL((k_quant_b128<BF16, F, true, false, true, 8>), grid, block, 0, stream, a);
  else if (row && col)
    hipLaunchKernelGGL((k_quant_b128<BF16, F, true, true, false, 8>), grid, block, 0, stream, a);
  else if (col)
    hipLaunchKernelGGL((k_quant_b128<BF16, F, false, true, false, 8>), grid, block, 0, stream, a);
  else if (thin)
    hipLaunchKernelGGL((k_quant_b128<BF16, F, true, false, false, 1>), grid, block, 0, stream, a);
  else
    hipLaunchKernelGGL((k_quant_b128<BF16, F, true, false, false, 8>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_quant_b128(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, int fmt, int rule,
                             bool tile, uint8_t* rc, int64_t ld_rc, float* rs, int64_t ld_rs, uint8_t* cc, int64_t ld_cc,
                             float* cs, int64_t ld_cs, const int* offsets, int experts, hipStream_t stream) {
  QuantArgs a{};
  a.src = src;
  a.rows = rows;
  a.cols = cols;
  a.ld = ld_src;
  a.rc = rc;
  a.ld_rc = ld_rc;
  a.rs = rs;
  a.ld_rs = ld_rs;
  a.cc = cc;
  a.ld_cc = ld_cc;
  a.cs = cs;
  a.ld_cs = ld_cs;
  a.offsets = offsets;
  a.experts = experts;
  a.rule = rule;
  a.blocks_c = (int)grouped_tiles(rows, offsets ? experts : 1, kB);
  a.vec = ((uintptr_t)src % 16 == 0) && (ld_src * (src_bf16 ? 2 : 4)) % 16 == 0;
  const bool row = rc != nullptr, col = cc != nullptr;
  if (src_bf16) return fmt == kE4M3 ? launch_f<1, kE4M3>(a, row, col, tile, stream) : launch_f<1, kE5M2>(a, row, col, tile, stream);
  return fmt == kE4M3 ? launch_f<0, kE4M3>(a, row, col, tile, stream) : launch_f<0, kE5M2>(a, row, col, tile, stream);
}

}  // namespace mxq
