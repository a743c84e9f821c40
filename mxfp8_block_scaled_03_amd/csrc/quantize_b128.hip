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
  int experts, rule, blocks_c;   // blocks_c: blocks that a line of cc and cs has room for
  int tiles_c;
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

// Lane q's value to all 16 lanes of its row of lanes.
__device__ __forceinline__ float bcast16(float v, int q) {
  const int x = __float_as_int(v);
  int r = x;
  switch (q) {   // row_newbcast:q; q is a constant after unrolling
    case 0: r = __builtin_amdgcn_update_dpp(0, x, 0x150, 0xF, 0xF, false); break;
    case 1: r = __builtin_amdgcn_update_dpp(0, x, 0x151, 0xF, 0xF, false); break;
    case 2: r = __builtin_amdgcn_update_dpp(0, x, 0x152, 0xF, 0xF, false); break;
    case 3: r = __builtin_amdgcn_update_dpp(0, x, 0x153, 0xF, 0xF, false); break;
    case 4: r = __builtin_amdgcn_update_dpp(0, x, 0x154, 0xF, 0xF, false); break;
    case 5: r = __builtin_amdgcn_update_dpp(0, x, 0x155, 0xF, 0xF, false); break;
    case 6: r = __builtin_amdgcn_update_dpp(0, x, 0x156, 0xF, 0xF, false); break;
    default: r = __builtin_amdgcn_update_dpp(0, x, 0x157, 0xF, 0xF, false); break;
  }
  return __int_as_float(r);
}

// Eight values times eight factors: two dwords of codes.
template <int F>
__device__ __forceinline__ uint2 encode8(const float v[8]) {
  uint32_t d[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    uint32_t p[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) p[e] = __float_as_uint(v[4 * h + e]);
    d[h] = mxblock::cvt2_f32<F>(0u, p[0], p[1], 1.0f, false);
    d[h] = mxblock::cvt2_f32<F>(d[h], p[2], p[3], 1.0f, true);
  }
  return make_uint2(d[0], d[1]);
}

// 0x7F in the first n of eight codes.
__device__ __forceinline__ uint2 nan_codes(int n) {
  const uint64_t m = n >= 8 ? ~0ull : n <= 0 ? 0ull : (1ull << (8 * n)) - 1;
  const uint64_t c = 0x7F7F7F7F7F7F7F7Full & m;
  return make_uint2((uint32_t)c, (uint32_t)(c >> 32));
}

// A thread's Q x 8 values, kept as they were loaded.
template <int BF16, int Q>
struct Values {
  uint32_t w[Q][BF16 ? 4 : 8];
  __device__ __forceinline__ float at(int q, int e) const {
    if (BF16) return __uint_as_float(e & 1 ? w[q][e >> 1] & 0xFFFF0000u : w[q][e >> 1] << 16);
    return __uint_as_float(w[q][e]);
  }
};

// Bits of the larger magnitude, of both halves of a dword for bf16.
template <int BF16>
__device__ __forceinline__ uint32_t larger(uint32_t m, uint32_t w) {
  return BF16 ? mxblock::pk_abs_max_bf16(m, w) : max(m, w & 0x7FFFFFFFu);
}

constexpr int kQuad = 4;   // waves

template <bool COL>
struct Shared {
  uint32_t wave_max[kQuad][COL ? kB : 1];
  __attribute__((aligned(16))) float factor[COL ? kB : 4];
  __attribute__((aligned(16))) uint8_t codes[COL ? kB * kB : 16];
};

// WHOLE: no row or column of the tile lies outside the matrix.
template <int BF16, int F, bool ROW, bool COL, bool TILE, int Q, bool WHOLE>
__device__ __forceinline__ void quantize_tile(const QuantArgs& a, Shared<COL>& sh, int tr, int bc, int64_t row0, int rows,
                                              int out_block) {
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int c = tid & 15, rg = tid >> 4;
  const int64_t col = (int64_t)bc * kB + 8 * c;
  const int cols = WHOLE ? 8 : (int)min((int64_t)8, a.cols - col);   // of this thread's eight, 0 or less past the end
  Values<BF16, Q> v;
  if (WHOLE || cols >= 8) {
    // (two or one 16-byte loads, whatever the alignment; rows past the last ask for it again, without a branch: 8192 x
    // 4096 of 16 experts of any lengths, both orientations, 38.6 us value by value, 28.0 so, 25.8
    // without experts; 64 experts 57.5 and 30.6; 4095 x 4001 fp32 by tiles 21.3 and 16.5)
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = Q * rg + q;
      const int64_t at = (row0 + (WHOLE ? r : min(r, rows - 1))) * a.ld + col;
      __builtin_memcpy(v.w[q], reinterpret_cast<const uint8_t*>(a.src) + at * (BF16 ? 2 : 4), sizeof v.w[q]);
    }
    if (!WHOLE) {
#pragma unroll
      for (int q = 0; q < Q; ++q)
#pragma unroll
        for (int e = 0; e < (BF16 ? 4 : 8); ++e) v.w[q][e] = Q * rg + q < rows ? v.w[q][e] : 0u;
    }
  } else {
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = Q * rg + q;
      const int64_t at = (row0 + r) * a.ld + col;
#pragma unroll
      for (int e = 0; e < (BF16 ? 4 : 8); ++e) v.w[q][e] = 0;
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (r < rows && e < cols) {
          if (BF16)
            v.w[q][e >> 1] |= (uint32_t)reinterpret_cast<const uint16_t*>(a.src)[at + e] << (16 * (e & 1));
          else
            v.w[q][e] = reinterpret_cast<const uint32_t*>(a.src)[at + e];
        }
    }
  }
  // maxima: of rows over a lane's values and 16 lanes, of columns over a thread's rows, 4 lanes and 4 waves
  uint32_t rmax[Q], cpk[BF16 ? 4 : 8];
#pragma unroll
  for (int e = 0; e < (BF16 ? 4 : 8); ++e) cpk[e] = 0;
#pragma unroll
  for (int q = 0; q < Q; ++q) {
    uint32_t m = 0;
#pragma unroll
    for (int e = 0; e < (BF16 ? 4 : 8); ++e) {
      m = larger<BF16>(m, v.w[q][e]);
      if (COL && !TILE) cpk[e] = larger<BF16>(cpk[e], v.w[q][e]);
    }
    rmax[q] = BF16 ? max(m << 16, m & 0xFFFF0000u) : m;
  }
  float tile_s = 1.0f, tile_r = 1.0f;
  bool tile_bad = false;
  if (TILE) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < Q; ++q) m = max(m, rmax[q]);
#pragma unroll
    for (int d = 1; d < 64; d <<= 1) m = max(m, (uint32_t)__shfl_xor((int)m, d, 64));
    if (lane == 0) sh.wave_max[wave][0] = m;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kQuad; ++w) m = max(m, sh.wave_max[w][0]);
    scale_of<F>(m, a.rule, tile_s, tile_r);
    tile_bad = m >= 0x7F800000u;
    if (tid == 0) a.rs[(int64_t)tr * a.ld_rs + bc] = tile_s;
  }
  if (COL && !TILE) {
    uint32_t cmax[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      cmax[e] = BF16 ? (e & 1 ? cpk[e >> 1] & 0xFFFF0000u : cpk[e >> 1] << 16) : cpk[e & (BF16 ? 3 : 7)];
      cmax[e] = max(cmax[e], (uint32_t)__shfl_xor((int)cmax[e], 16, 64));
      cmax[e] = max(cmax[e], (uint32_t)__shfl_xor((int)cmax[e], 32, 64));
    }
    if (lane < 16) {
      *reinterpret_cast<uint4*>(&sh.wave_max[wave][8 * c]) = make_uint4(cmax[0], cmax[1], cmax[2], cmax[3]);
      *reinterpret_cast<uint4*>(&sh.wave_max[wave][8 * c + 4]) = make_uint4(cmax[4], cmax[5], cmax[6], cmax[7]);
    }
    __syncthreads();
    // a thread a column: its scale, and the factor for all (NaN where the block is to be NaN)
    if (tid < kB) {
      uint32_t m = 0;
#pragma unroll
      for (int w = 0; w < kQuad; ++w) m = max(m, sh.wave_max[w][tid]);
      float s, f;
      scale_of<F>(m, a.rule, s, f);
      sh.factor[tid] = m >= 0x7F800000u ? s : f;
      if (WHOLE || (int64_t)bc * kB + tid < a.cols) a.cs[(int64_t)out_block * a.ld_cs + (int64_t)bc * kB + tid] = s;
    }
  }
  if (ROW) {
    // a lane a row: of the 16 lanes of the same Q rows, lane q divides for row q, and all of them take its factor
    float s = tile_s, f = tile_r;
    bool bad = tile_bad;
    if (!TILE) {
#pragma unroll
      for (int q = 0; q < Q; ++q) rmax[q] = row16_max(rmax[q]);
      uint32_t m = rmax[0];
#pragma unroll
      for (int q = 1; q < Q; ++q) m = c == q ? rmax[q] : m;
      scale_of<F>(m, a.rule, s, f);
      bad = m >= 0x7F800000u;
      if (c < Q && (WHOLE || Q * rg + c < rows)) a.rs[(int64_t)bc * a.ld_rs + row0 + Q * rg + c] = s;
      if (bad) f = s;
    }
    const bool any_bad = __any(bad);
#pragma unroll
    for (int q = 0; q < Q; ++q) {
      const int r = Q * rg + q;
      float fq = f;
      if (!TILE && Q > 1) fq = bcast16(f, q);
      float x[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = v.at(q, e) * fq;
      uint2 d = encode8<F>(x);
      if (any_bad && (tile_bad || (!TILE && fq != fq))) d = nan_codes(cols);
      if (WHOLE || r < rows) *reinterpret_cast<uint2*>(a.rc + (row0 + r) * a.ld_rc + (int64_t)bc * kB + 8 * c) = d;
    }
  }
  if (COL) {
    float f[8];
    bool any_bad = tile_bad;
    if (TILE) {
#pragma unroll
      for (int e = 0; e < 8; ++e) f[e] = tile_r;
    } else {
      __syncthreads();
      const float4 lo = *reinterpret_cast<const float4*>(&sh.factor[8 * c]), hi = *reinterpret_cast<const float4*>(&sh.factor[8 * c + 4]);
      f[0] = lo.x, f[1] = lo.y, f[2] = lo.z, f[3] = lo.w, f[4] = hi.x, f[5] = hi.y, f[6] = hi.z, f[7] = hi.w;
      const float sum = (lo.x + lo.y) + (lo.z + lo.w) + (hi.x + hi.y) + (hi.z + hi.w);   // NaN if one of them is
      any_bad = __any(sum != sum);
    }
    // the eight codes of column 8 c + j, rows 8 rg .. 8 rg + 7, as an 8-byte word.  LDS row 8 c + (j ^ (c & 1))
    // of 16 words, word rg ^ (c & 14): the 32 lanes that write together touch every bank once.
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      float x[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) x[q] = v.at(q & (Q - 1), j) * f[j];
      uint2 d = encode8<F>(x);
      if (any_bad && (tile_bad || f[j] != f[j])) d = nan_codes(WHOLE ? 8 : rows - 8 * rg);
      *reinterpret_cast<uint2*>(sh.codes + (8 * c + (j ^ (c & 1))) * kB + 8 * (rg ^ (c & 14))) = d;
    }
    __syncthreads();
#pragma unroll
    for (int it = 0; it < 4; ++it) {
      const int k = 32 * it + (tid >> 3), p = tid & 7, kc = k >> 3;   // column k, rows 16 p .. 16 p + 15
      const uint4 u = *reinterpret_cast<const uint4*>(sh.codes + (8 * kc + ((k & 7) ^ (kc & 1))) * kB + 8 * ((2 * p) ^ (kc & 14)));
      if (WHOLE || (int64_t)bc * kB + k < a.cols)
        *reinterpret_cast<uint4*>(a.cc + ((int64_t)bc * kB + k) * a.ld_cc + (int64_t)out_block * kB + 16 * p) = u;
    }
  }
}

// Q rows a thread (8, or 1 where rows alone are wanted and few tiles of 128 rows would leave the card empty).
template <int BF16, int F, bool ROW, bool COL, bool TILE, int Q>
__global__ __launch_bounds__(256) void k_quant_b128(const QuantArgs a) {
  constexpr int kRows = 16 * Q;
  __shared__ Shared<COL> sh;
  const int bc = blockIdx.x % a.tiles_c, tr = blockIdx.x / a.tiles_c;
  int64_t row0 = (int64_t)tr * kRows;
  int rows = (int)min((int64_t)kRows, a.rows - row0);
  if (COL && a.offsets) {
    const Group g = find_group(a.offsets, a.experts, (int)a.rows, kB, 1, tr);
    if (g.e < 0 || tr >= a.blocks_c) return;
    row0 = g.row0 + kB * g.tile;
    rows = min(kB, g.rows - kB * g.tile);
  }
  if (rows == kRows && ((int64_t)bc + 1) * kB <= a.cols)
    quantize_tile<BF16, F, ROW, COL, TILE, Q, true>(a, sh, tr, bc, row0, rows, tr);
  else
    quantize_tile<BF16, F, ROW, COL, TILE, Q, false>(a, sh, tr, bc, row0, rows, tr);
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
  const bool row = rc != nullptr, col = cc != nullptr;
  if (src_bf16) return fmt == kE4M3 ? launch_f<1, kE4M3>(a, row, col, tile, stream) : launch_f<1, kE5M2>(a, row, col, tile, stream);
  return fmt == kE4M3 ? launch_f<0, kE4M3>(a, row, col, tile, stream) : launch_f<0, kE5M2>(a, row, col, tile, stream);
}

}  // namespace mxq
