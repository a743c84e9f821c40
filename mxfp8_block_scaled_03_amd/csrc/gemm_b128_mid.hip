// gemm_b128_mid.hip -- the product in blocks of 128 by tiles of 64 x 64 and 128 x 128, where 256 x 256 would leave the
// card, or the tiles of uneven experts, half empty.
//
// WM x WN waves share a tile (KS = 2: twice, every other step for each half, whose sums meet in LDS); a step is one
// block of K, and S steps' codes lie in LDS, so that the loads of a step have S - U steps to arrive.  Lines, pieces,
// fragments and sums as in gemm_b128_tile.hip; a step is short, so rounds of U steps have one barrier: the one that says
// that a round's codes are there also says that nobody reads the round before it any more, whose place is filled next.
#include "gemm_b128.hpp"

namespace mxq {
namespace {

template <int TM, int TN, int WM, int WN, int KS, int S, int U>
struct Mid {
  static constexpr int kWaves = WM * WN * KS, kThreads = 64 * kWaves;
  static constexpr int kX = TM * kB, kStage = (TM + TN) * kB;
  static constexpr int kOffScale = S * kStage, kScaleSlot = 4 * (TM + TN);
  static constexpr int kLds = kOffScale + S * kScaleSlot;
  static constexpr int kLoadsX = TM / 8 / kWaves, kLoadsW = TN / 8 / kWaves;      // instructions a wave and step
  static constexpr int kLoads = kLoadsX + kLoadsW + 1;
  static constexpr int FM = TM / WM / 16, FN = TN / WN / 16;
  static constexpr int kRegion = kOffScale / (WM * WN);
  static_assert(S % U == 0 && S >= 2 * U && U % KS == 0, "rounds of U steps, of U / KS for each wave");
  static_assert(KS <= 2 && 1024 * FM * FN <= kRegion, "the second waves' sums");
  static_assert((TM + TN) / 64 <= kWaves, "a wave for each 64 scales");
};

template <int FX, int FW, bool EXACT, bool WLINE, int TM, int TN, int WM, int WN, int KS, int S, int U>
__global__ __launch_bounds__(64 * WM * WN * KS, 2) void k_gemm_b128_mid(const GemmB128 a) {
  using C = Mid<TM, TN, WM, WN, KS, S, U>;
  constexpr int FM = C::FM, FN = C::FN;
  const B128Tile t = b128_tile<TM, TN, WLINE>(a, workgroup_at(blockIdx.x, blockIdx.y));
  if (!t.any) return;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
  const int nb = t.nb;
  const int rows_x = min(TM, t.m), rows_w = min(TN, t.n);
  const uint64_t x_base = (uint64_t)(uintptr_t)t.x, w_base = (uint64_t)(uintptr_t)t.w;
  const uint32_t line_bytes = (uint32_t)nb * kB;
  const uint32_t x_bytes = (uint32_t)((rows_x - 1) * a.ld_x) + line_bytes;
  const uint32_t w_bytes = (uint32_t)((rows_w - 1) * a.ld_w) + line_bytes;
  // instruction n of a wave: lines 8 (wid L + n) + lane / 8; the piece there follows from the line
  const int sub = lane >> 3, x_line = 8 * C::kLoadsX * wid, w_line = 8 * C::kLoadsW * wid;
  auto piece = [&](int line0, int n) { return (uint32_t)(((lane & 7) ^ ((((line0 >> 1) & 4) + 4 * n + (sub >> 1)) & 7)) << 4); };
  const uint32_t vx = (uint32_t)((x_line + sub) * a.ld_x), vw = (uint32_t)((w_line + sub) * a.ld_w);
  const uint32_t x8 = (uint32_t)(8 * a.ld_x), w8 = (uint32_t)(8 * a.ld_w);
  const uint32_t lds_x = lds0 + (uint32_t)x_line * kB, lds_w = lds0 + C::kX + (uint32_t)w_line * kB;
  // scales: 64 lines a wave, X's first, then W's; waves past them load nothing
  const bool sx_wave = wid < TM / 64, s_wave = wid < (TM + TN) / 64;
  const uint64_t s_base = (uint64_t)(uintptr_t)(sx_wave ? t.xs : t.ws);
  const int s_line = 64 * (sx_wave ? wid : wid - TM / 64) + lane;
  const int64_t s_step = 4 * (sx_wave ? a.ld_xs : a.ws_k);
  uint32_t s_voff, s_bytes;
  if (sx_wave || WLINE) {
    s_voff = 4u * (uint32_t)s_line;
    s_bytes = 4u * (uint32_t)(sx_wave ? rows_x : rows_w);
  } else {
    s_voff = 0u;                       // a tile of W's scales holds the whole of TN <= 128 columns
    s_bytes = 4u;
  }
  const uint32_t lds_s = lds0 + C::kOffScale + 256u * (uint32_t)wid;

  auto issue = [&](int s, int slot) {
    const bool live = s < nb;
    const uint32_t kb = live ? (uint32_t)s * kB : 0u;
    const v4i rx = rsrc_of(x_base + kb, live ? x_bytes - kb : 0u), rw = rsrc_of(w_base + kb, live ? w_bytes - kb : 0u);
    const uint32_t so = (uint32_t)slot * C::kStage;
#pragma unroll
    for (int n = 0; n < C::kLoadsX; ++n) dma16(lds_x + so + 1024u * n, vx + n * x8 + piece(x_line, n), rx);
#pragma unroll
    for (int n = 0; n < C::kLoadsW; ++n) dma16(lds_w + so + 1024u * n, vw + n * w8 + piece(w_line, n), rw);
    if (s_wave) {
      const v4i rs = rsrc_of(s_base + (live ? (uint64_t)(s * s_step) : 0u), live ? s_bytes : 0u);
      dma4(lds_s + (uint32_t)slot * C::kScaleSlot, s_voff, rs);
    }
  };

  const int part = wid / (WM * WN), m0 = 16 * FM * (wid / WN % WM), n0 = 16 * FN * (wid % WN);
  const uint32_t frag = (uint32_t)i * kB + (uint32_t)((g ^ (i >> 1)) << 4);
  const uint32_t rx = (uint32_t)m0 * kB + frag, rw = C::kX + (uint32_t)n0 * kB + frag;
  const uint32_t rsx = C::kOffScale + 4u * (uint32_t)(m0 + i);
  const uint32_t rsw = C::kOffScale + 4u * (uint32_t)(TM + n0 + (WLINE ? 4 * g : 0));
  auto fragment = [&](uint32_t at, int f) {
    const v4i lo = lds16(at, 2048 * f), hi = lds16(at ^ 64u, 2048 * f);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  v4f acc[FM][FN];
#pragma unroll
  for (int f = 0; f < FM; ++f)
#pragma unroll
    for (int j = 0; j < FN; ++j) acc[f][j] = {0.0f, 0.0f, 0.0f, 0.0f};

#pragma unroll
  for (int s = 0; s < S - U; ++s) issue(s, s);
  int first = 0;   // the slot of the round's first step
  for (int s0 = 0; s0 < nb; s0 += U) {
    // the round's U steps have arrived: all but the newest S - 2 U steps' loads (waves without scales have fewer)
    if (s_wave)
      wait_vm<(S - 2 * U) * C::kLoads>();
    else
      wait_vm<(S - 2 * U) * (C::kLoads - 1)>();
    lds_barrier();
#pragma unroll
    for (int u = 0; u < U; ++u) issue(s0 + S - U + u, (first == 0 ? S : first) - U + u);
#pragma unroll
    for (int u = 0; u < U; u += KS) {
      const int slot = first + u + part;
      const uint32_t so = (uint32_t)slot * C::kStage, ss = (uint32_t)slot * C::kScaleSlot;
      v8i w[FN];
      Wide ww[FN];
#pragma unroll
      for (int j = 0; j < FN; ++j) {
        w[j] = fragment(rw + so, j);
        if (EXACT) ww[j] = widen<FW>(w[j]);
      }
      float sw1 = 0.0f;
      v4f sw[FN];
      if (WLINE) {
#pragma unroll
        for (int j = 0; j < FN; ++j) sw[j] = *reinterpret_cast<const v4f*>(smem + rsw + ss + 64 * j);
      } else {
        sw1 = *reinterpret_cast<const float*>(smem + rsw + ss);
      }
#pragma unroll
      for (int f = 0; f < FM; ++f) {
        const v8i x = fragment(rx + so, f);
        const float sx = *reinterpret_cast<const float*>(smem + rsx + ss + 64 * f);
        v4f d[FN];
        if (EXACT) {
          const Wide xw = widen<FX>(x);
#pragma unroll
          for (int j = 0; j < FN; ++j) d[j] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < FN; ++j) d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[j].p[q], xw.p[q], d[j], 0, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < FN; ++j) d[j] = block_fp8<FX, FW>(w[j], x);
        }
#pragma unroll
        for (int j = 0; j < FN; ++j) {
          const float sc = sx * sw1;
#pragma unroll
          for (int r = 0; r < 4; ++r) acc[f][j][r] = __builtin_fmaf(d[j][r], WLINE ? sx * sw[j][r] : sc, acc[f][j][r]);
        }
      }
    }
    first = first == S - U ? 0 : first + U;
  }
  wait_vm<0>();
  lds_barrier();
  if (KS == 2) {
    // the second waves' sums to the first, through what will be those's own staging
    v4f* const sums = reinterpret_cast<v4f*>(smem + C::kRegion * (wid - part * WM * WN)) + lane;
    if (part != 0) {
#pragma unroll
      for (int f = 0; f < FM; ++f)
#pragma unroll
        for (int j = 0; j < FN; ++j) sums[64 * (f * FN + j)] = acc[f][j];
    }
    lds_barrier();
    if (part != 0) return;
#pragma unroll
    for (int f = 0; f < FM; ++f)
#pragma unroll
      for (int j = 0; j < FN; ++j) acc[f][j] += sums[64 * (f * FN + j)];
  }
  epilogue<FM, FN, C::kRegion>(a, t, acc, wid, lane, m0, n0);
}

template <int FX, int FW, bool EXACT, bool WLINE, int TM, int TN, int WM, int WN, int KS, int S, int U>
hipError_t launch_t(const GemmB128& a, hipStream_t stream) {
  using C = Mid<TM, TN, WM, WN, KS, S, U>;
  static bool set[64] = {false};
  auto kern = k_gemm_b128_mid<FX, FW, EXACT, WLINE, TM, TN, WM, WN, KS, S, U>;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!set[dev]) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, C::kLds);
    if (e != hipSuccess) return e;
    set[dev] = true;
  }
  const Grid grid = grid_of(gemm_b128_tiles(a, TM, TN));
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(C::kThreads), C::kLds, stream, a);
  return hipGetLastError();
}

template <int FX, int FW, bool EXACT, bool WLINE>
hipError_t launch_p(const GemmB128& a, const GemmB128Plan& p, hipStream_t s) {
  // Four steps in LDS: a workgroup's loads have three steps (tiles of 64: a round of two) to arrive.  Where there are
  // more tiles than that leaves room for at once, two steps and twice the workgroups on a CU (2048 x 4096 x
  // 4096: 51 us with four steps, 43 with two; 1024 rows 27 and 31).
  const int64_t cus = device_cu_count(), tiles = gemm_b128_tiles(a, p.tile_m, p.tile_n);
  // Tiles of 64 that leave no CU two: twice the waves, for alternate steps each (1000 x 1000 x 4001 exact 20.0 -> 17.8
  // us, 256 x 4096 x 4096 fp8 13.3 -> 11.6; with two tiles a CU 11.3 and 12.1).  Then codes arrive at 9.4 TB/s, and
  // eight steps in LDS make it slower (12.7 for 11.6).
  if (p.tile_m == 64 && tiles <= cus) return launch_t<FX, FW, EXACT, WLINE, 64, 64, 2, 2, 2, 4, 2>(a, s);
  if (p.tile_m == 64)
    return tiles <= 2 * cus ? launch_t<FX, FW, EXACT, WLINE, 64, 64, 2, 2, 1, 4, 2>(a, s)
                            : launch_t<FX, FW, EXACT, WLINE, 64, 64, 2, 2, 1, 2, 1>(a, s);
  return tiles <= cus ? launch_t<FX, FW, EXACT, WLINE, 128, 128, 2, 4, 1, 4, 1>(a, s)
                      : launch_t<FX, FW, EXACT, WLINE, 128, 128, 2, 4, 1, 2, 1>(a, s);
}

template <int FX, int FW>
hipError_t launch_f(const GemmB128& a, const GemmB128Plan& p, hipStream_t s) {
  if (a.exact) return a.w_line ? launch_p<FX, FW, true, true>(a, p, s) : launch_p<FX, FW, true, false>(a, p, s);
  return a.w_line ? launch_p<FX, FW, false, true>(a, p, s) : launch_p<FX, FW, false, false>(a, p, s);
}

}  // namespace

hipError_t launch_gemm_b128_mid(const GemmB128& a, const GemmB128Plan& p, hipStream_t s) {
  if (a.x_fmt == kE4M3) return a.w_fmt == kE4M3 ? launch_f<0, 0>(a, p, s) : launch_f<0, 1>(a, p, s);
  return a.w_fmt == kE4M3 ? launch_f<1, 0>(a, p, s) : launch_f<1, 1>(a, p, s);
}

}  // namespace mxq
