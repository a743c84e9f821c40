// gemm_b128_rows.hip -- the product in blocks of 128 by small tiles: few rows (a decoding step, a few tokens an
// expert), and outputs too small to fill the card with 256 x 256 tiles.
//
// Bound by the weights' bytes and by latency.  A wave owns 16 MT x 16 NT outputs.  Where there are few tiles
// (WK = 8) eight waves share them along K: wave v takes blocks v, v + 8, ..., so that the eight together read
// 1 KiB runs of each line; their sums meet in LDS, are added in the waves' order, and finished by all
// threads.  Where there are many (WK = 1: experts of a
// row or two) each of four waves has a tile of its own, side by side along N,
// and all of K.  Codes come straight from memory into the fragments' registers, U blocks ahead: a block's
// registers are refilled as soon as they have been read.
#include "gemm_b128.hpp"

namespace mxq {
namespace {

template <int FX, int FW, bool EXACT, bool WLINE, int MT, int NT, int U, int WK>
struct RowsWave {
  __amdgpu_buffer_rsrc_t rx, rw, rsx, rsw;
  uint32_t vx, vw;
  int64_t ld_xs, ws_k;
  uint32_t x16, w16;
  int nb, i, g;
  // U blocks' codes and scales, each refilled with the block U further on as soon as it has been read
  v4i x[U][MT][2], w[U][NT][2];
  float sx[U][MT];
  v4f sw[U][WLINE ? NT : 1];

  // past the last block: an offset past every range (each below 2^31), for which loads give zeros
  __device__ __forceinline__ uint32_t dead(int b) const { return b < nb ? 0u : 0x80000000u; }
  __device__ __forceinline__ void load_w(int u, int b) {
    const uint32_t at = (uint32_t)b * kB, d = dead(b);
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        w[u][j][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)((vw + j * w16 + 64 * h + at) | d), 0, 0));
    const uint32_t wa = (uint32_t)(4 * (b * ws_k + (WLINE ? 4 * g : 0)));
    if (WLINE) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
        sw[u][j] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsw, (int)((wa + 64 * j) | d), 0, 0));
    } else {
      sw[u][0][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsw, (int)(wa | d), 0, 0));
    }
  }
  __device__ __forceinline__ void load_x(int u, int f, int b) {
    const uint32_t at = (uint32_t)b * kB, d = dead(b);
#pragma unroll
    for (int h = 0; h < 2; ++h)
      x[u][f][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)((vx + f * x16 + 64 * h + at) | d), 0, 0));
    sx[u][f] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsx, (int)((uint32_t)(4 * (b * ld_xs + i) + 64 * f) | d), 0, 0));
  }
  __device__ __forceinline__ void fill(int b0) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      load_w(u, b0 + WK * u);
#pragma unroll
      for (int f = 0; f < MT; ++f) load_x(u, f, b0 + WK * u);
    }
  }
  // U blocks from b0 on; MORE: there are blocks behind them, which take their places
  template <bool MORE>
  __device__ __forceinline__ void multiply(int b0, v4f acc[MT][NT]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int next = b0 + WK * (U + u);
      v8i wu[NT];
      Wide ww[NT];
      v4f su[WLINE ? NT : 1];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        wu[j] = __builtin_shufflevector(w[u][j][0], w[u][j][1], 0, 1, 2, 3, 4, 5, 6, 7);
        if (EXACT) ww[j] = widen<FW>(wu[j]);
        if (WLINE || j == 0) su[j] = sw[u][j];
      }
      if (MORE && EXACT) load_w(u, next);
#pragma unroll
      for (int f = 0; f < MT; ++f) {
        const v8i xu = __builtin_shufflevector(x[u][f][0], x[u][f][1], 0, 1, 2, 3, 4, 5, 6, 7);
        const float sxu = sx[u][f];
        v4f d[NT];
        if (EXACT) {
          const Wide xw = widen<FX>(xu);
          if (MORE) load_x(u, f, next);
#pragma unroll
          for (int j = 0; j < NT; ++j) d[j] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < NT; ++j) d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[j].p[q], xw.p[q], d[j], 0, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < NT; ++j) d[j] = block_fp8<FX, FW>(wu[j], xu);
          if (MORE) load_x(u, f, next);
        }
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[f][j][r] = __builtin_fmaf(d[j][r], sxu * (WLINE ? su[j][r] : su[0][0]), acc[f][j][r]);
      }
      if (MORE && !EXACT) load_w(u, next);
    }
  }
};

// Four outputs of row m from column n on (both of the tile), `left` of them inside.
__device__ __forceinline__ void store4(const GemmB128& a, const B128Tile& t, v4f s, int m, int n, int left) {
#pragma unroll
  for (int r = 0; r < 4; ++r) s[r] = finish(s[r], a.alpha, a.bias && r < left ? a.bias[t.n0 + n + r] : -0.0f, a.act);
  const int64_t at = t.y + (int64_t)m * a.ld_y + n;
  if (a.y_bf16) {
    uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + at;
    const v2u d = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
    if (left >= 4) {
      __builtin_memcpy(y, &d, 8);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) y[r] = (uint16_t)(d[r >> 1] >> (16 * (r & 1)));
    }
  } else {
    float* y = reinterpret_cast<float*>(a.y) + at;
    if (left >= 4) {
      __builtin_memcpy(y, &s, 16);
    } else {
#pragma unroll
      for (int r = 0; r < 4; ++r)
        if (r < left) y[r] = s[r];
    }
  }
}

constexpr int waves_of(int wk) { return wk == 1 ? 4 : wk; }

template <int FX, int FW, bool EXACT, bool WLINE, int MT, int NT, int WK>
__global__ __launch_bounds__(64 * waves_of(WK), 2) void k_gemm_b128_rows(const GemmB128 a) {
  constexpr int kThreads = 64 * waves_of(WK), WN = waves_of(WK) / WK;
  // (blocks in registers; more are no faster: 16 rows with eight 8.1 us for 7.0, 32 with four 8.7 for 9.0 but 64 x 2048 x
  // 1024 5.6 for 4.8, 64 x 32 with two 14.5 for 15.0 but exact, where they spill, 20 for 14.7)
  constexpr int U = MT + NT <= 2 ? 4 : MT + NT <= 4 ? 2 : 1;
  B128Tile t = b128_tile<16 * MT, 16 * NT * WN, WLINE, WK != 1>(a, workgroup_at(blockIdx.x, blockIdx.y));
  if (!t.any) return;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wk = wid % WK;
  if (WN > 1) {
    // this wave's columns (those of the workgroup lie in one tile of W's scales)
    static_assert(kB % (16 * NT * WN) == 0, "a workgroup's columns end where a tile of scales does, or before");
    const int n = 16 * NT * (wid / WK);
    if (n >= t.n) return;
    t.w += n * a.ld_w;
    if (WLINE) t.ws += n;
    t.y += n;
    t.n -= n;
    t.n0 += n;
  }
  const int rows_x = min(16 * MT, t.m), rows_w = min(16 * NT, t.n);
  using Wave = RowsWave<FX, FW, EXACT, WLINE, MT, NT, U, WK>;
  Wave v;
  v.i = lane & 15;
  v.g = lane >> 4;
  v.nb = t.nb;
  const uint32_t line_bytes = (uint32_t)t.nb * kB;
  v.rx = make_rsrc(t.x, t.nb ? (uint32_t)((rows_x - 1) * a.ld_x) + line_bytes : 0u);
  v.rw = make_rsrc(t.w, t.nb ? (uint32_t)((rows_w - 1) * a.ld_w) + line_bytes : 0u);
  v.vx = (uint32_t)(v.i * a.ld_x) + 16u * v.g;
  v.vw = (uint32_t)(v.i * a.ld_w) + 16u * v.g;
  v.x16 = (uint32_t)(16 * a.ld_x);
  v.w16 = (uint32_t)(16 * a.ld_w);
  v.ld_xs = a.ld_xs;
  v.ws_k = a.ws_k;
  v.rsx = make_rsrc(t.xs, t.nb ? (uint32_t)(4 * ((t.nb - 1) * a.ld_xs + rows_x)) : 0u);
  v.rsw = make_rsrc(t.ws, t.nb ? (uint32_t)(4 * ((t.nb - 1) * a.ws_k + (WLINE ? rows_w : 1))) : 0u);

  v4f acc[MT][NT];
#pragma unroll
  for (int f = 0; f < MT; ++f)
#pragma unroll
    for (int j = 0; j < NT; ++j) acc[f][j] = {0.0f, 0.0f, 0.0f, 0.0f};
  constexpr int step = WK * U;
  int b = wk;
  v.fill(b);
  for (; b + step < t.nb; b += step) v.template multiply<true>(b, acc);
  v.template multiply<false>(b, acc);
  if (WK == 1) {
#pragma unroll
    for (int f = 0; f < MT; ++f)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        const int m = 16 * f + v.i, n = 16 * j + 4 * v.g;
        if (m < rows_x && n < rows_w) store4(a, t, acc[f][j], m, n, rows_w - n);
      }
    return;
  }
  v4f* part = reinterpret_cast<v4f*>(smem);
#pragma unroll
  for (int f = 0; f < MT; ++f)
#pragma unroll
    for (int j = 0; j < NT; ++j) part[(wid * MT * NT + f * NT + j) * 64 + lane] = acc[f][j];
  __syncthreads();
  for (int o = threadIdx.x; o < MT * NT * 64; o += kThreads) {
    v4f s = part[o];
#pragma unroll
    for (int w = 1; w < WK; ++w) {
      const v4f e = part[w * MT * NT * 64 + o];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] += e[r];
    }
    const int l = o & 63, f = (o >> 6) / NT, j = (o >> 6) % NT;
    const int m = 16 * f + (l & 15), n = 16 * j + 4 * (l >> 4);
    if (m < rows_x && n < rows_w) store4(a, t, s, m, n, rows_w - n);
  }
}

template <int FX, int FW, bool EXACT, bool WLINE, int MT, int NT, int WK>
hipError_t launch_t(const GemmB128& a, hipStream_t stream) {
  constexpr int waves = waves_of(WK), lds = WK == 1 ? 0 : WK * MT * NT * 1024;
  auto kern = k_gemm_b128_rows<FX, FW, EXACT, WLINE, MT, NT, WK>;
  static_assert(lds <= 65536, "no more than a launch may have unasked");
  const Grid grid = grid_of(gemm_b128_tiles(a, 16 * MT, 16 * NT * (waves / WK)));
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(64 * waves), lds, stream, a);
  return hipGetLastError();
}

template <int FX, int FW, bool EXACT, bool WLINE>
hipError_t launch_p(const GemmB128& a, const GemmB128Plan& p, hipStream_t s) {
  // the plans of gemm_b128_plan, and no others
  if (p.waves == 1) return launch_t<FX, FW, EXACT, WLINE, 1, 1, 1>(a, s);
  if (p.tile_m == 16) return launch_t<FX, FW, EXACT, WLINE, 1, 1, 8>(a, s);
  if (p.tile_m == 32) return launch_t<FX, FW, EXACT, WLINE, 2, 1, 8>(a, s);
  return launch_t<FX, FW, EXACT, WLINE, 4, 2, 8>(a, s);
}

template <int FX, int FW>
hipError_t launch_f(const GemmB128& a, const GemmB128Plan& p, hipStream_t s) {
  if (a.exact) return a.w_line ? launch_p<FX, FW, true, true>(a, p, s) : launch_p<FX, FW, true, false>(a, p, s);
  return a.w_line ? launch_p<FX, FW, false, true>(a, p, s) : launch_p<FX, FW, false, false>(a, p, s);
}

}  // namespace

hipError_t launch_gemm_b128_rows(const GemmB128& a, const GemmB128Plan& p, hipStream_t s) {
  if (a.x_fmt == kE4M3) return a.w_fmt == kE4M3 ? launch_f<0, 0>(a, p, s) : launch_f<0, 1>(a, p, s);
  return a.w_fmt == kE4M3 ? launch_f<1, 0>(a, p, s) : launch_f<1, 1>(a, p, s);
}

}  // namespace mxq
