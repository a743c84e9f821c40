// gemm_b128_tile.hip -- the product in blocks of 128 by 256 x 256 tiles.
//
// Eight waves, two to a SIMD; a wave owns 128 (m) x 64 (n) outputs: 8 x 4 tiles of 16 x 16, 128 accumulators.
// A step is one block of K: 256 lines of X and of W, 128 bytes each, 64 KiB, and two steps' codes lie in LDS.
// 16-byte piece p of line r is stored at p ^ ((r >> 1) & 7), which spreads the 16 lines of a fragment over all
// banks.  In a step a wave reads its fragments of W (32 registers) and then one fragment of X after the other;
// each meets the four of W from zero, and the 16 sums go to the accumulators by a fused multiply-add with sx sw.
//
// Codes move by buffer_load .. lds, eight lines of whole 128-byte lines an instruction.  Their places free
// up in two parts: at the middle of a step every wave has read W and the first half of its X lines, and at
// the end the second half.  What the middle frees is filled for the step after the next, which waits for
// it one and a half steps later, and so for the second half, which is first read in the middle of its step: 96 KiB are on their way
// on average with 128 KiB of LDS.  Every wave issues the same loads each step (two of the second half
// of X, then four of W, two of the first half of X and one of scales), so every wait is for all but the newest 9.
//
// Scales: waves 0-3 bring 64 lines' each of X, waves 4-7 of W, one dword a lane, into one of four slots; where W has tiles, each
// line's lane asks for its tile's.
#include "gemm_b128.hpp"

namespace mxq {
namespace {

constexpr int kThreads = 512;
constexpr int kTile = 256;
constexpr int kSide = kTile * kB;               // one operand's codes of a step: 32 KiB
constexpr int kStage = 2 * kSide;
constexpr int kOffScale = 2 * kStage;
constexpr int kScaleSlot = 2 * kTile * 4;       // X, then W
constexpr int kLds = kOffScale + 4 * kScaleSlot;   // 136 KiB
constexpr int kWaveOut = 16384;                 // a wave's staging of the epilogue, in the code stages

template <int FX, int FW, bool EXACT, bool WLINE>
__global__ __launch_bounds__(kThreads, 2) void k_gemm_b128(const GemmB128 a) {
  const B128Tile t = b128_tile<kTile, kTile, WLINE>(a, workgroup_at(blockIdx.x, blockIdx.y));
  if (!t.any) return;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int gp = wid >> 2, wq = wid & 3;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem;
  const int nb = t.nb;
  const int rows_x = min(kTile, t.m), rows_w = min(kTile, t.n);

  // ---- loads: instruction n of a wave covers lines base + 8 n + lane / 8, piece lane & 7 there holding piece
  //      (lane & 7) ^ ((line >> 1) & 7).  X: lines 16 wid' + 8 n of each half (wid' = wid & 3, the halves of
  //      wave group wid >> 2); W: lines 32 wid + 8 n.
  const uint64_t x_base = (uint64_t)(uintptr_t)t.x, w_base = (uint64_t)(uintptr_t)t.w;
  const uint32_t line_bytes = (uint32_t)nb * kB;
  const uint32_t x_bytes = (uint32_t)((rows_x - 1) * a.ld_x) + line_bytes;
  const uint32_t w_bytes = (uint32_t)((rows_w - 1) * a.ld_w) + line_bytes;
  const int sub = lane >> 3;
  const uint32_t piece0 = (uint32_t)(((lane & 7) ^ (sub >> 1)) << 4);   // line base a multiple of 16; else piece ^ 4
  const int x_line = 128 * gp + 16 * wq, w_line = 32 * wid;
  const uint32_t vx = (uint32_t)((x_line + sub) * a.ld_x), vw = (uint32_t)((w_line + sub) * a.ld_w);
  const uint32_t x8 = (uint32_t)(8 * a.ld_x), w8 = (uint32_t)(8 * a.ld_w);
  const uint32_t lds_x = lds0 + (uint32_t)x_line * kB, lds_w = lds0 + kSide + (uint32_t)w_line * kB;
  // scales: this wave's 64 lines
  const bool sx_wave = wid < 4;
  const uint64_t s_base = (uint64_t)(uintptr_t)(sx_wave ? t.xs : t.ws);
  const int s_line = 64 * (wid & 3) + lane;
  const int64_t s_step = 4 * (sx_wave ? a.ld_xs : a.ws_k);
  uint32_t s_voff, s_bytes;
  if (sx_wave || WLINE) {
    s_voff = 4u * (uint32_t)s_line;
    s_bytes = 4u * (uint32_t)(sx_wave ? rows_x : rows_w);
  } else {
    const int last = (rows_w - 1) / kB;
    s_voff = (uint32_t)(4 * a.ws_n * min(s_line / kB, last));
    s_bytes = (uint32_t)(4 * a.ws_n * last) + 4u;
  }
  const uint32_t lds_s = lds0 + kOffScale + (uint32_t)(sx_wave ? 0 : 4 * kTile) + 256u * (uint32_t)(wid & 3);

  auto issue_x = [&](int s, int half) {
    const bool live = s < nb;
    const uint32_t kb = live ? (uint32_t)s * kB : 0u;
    const v4i r = rsrc_of(x_base + kb, live ? x_bytes - kb : 0u);
    const uint32_t at = lds_x + (uint32_t)(s & 1) * kStage + (uint32_t)(64 * half) * kB;
    const uint32_t v = vx + (half ? 8 * x8 : 0u);
    dma16(at, v + piece0, r);
    dma16(at + 8 * kB, v + x8 + (piece0 ^ 64), r);
  };
  auto issue_w = [&](int s) {
    const bool live = s < nb;
    const uint32_t kb = live ? (uint32_t)s * kB : 0u;
    const v4i r = rsrc_of(w_base + kb, live ? w_bytes - kb : 0u);
    const uint32_t at = lds_w + (uint32_t)(s & 1) * kStage;
#pragma unroll
    for (int n = 0; n < 4; ++n) dma16(at + n * 8 * kB, vw + n * w8 + (n & 1 ? piece0 ^ 64 : piece0), r);
  };
  auto issue_s = [&](int s) {
    const bool live = s < nb;
    const v4i r = rsrc_of(s_base + (live ? (uint64_t)(s * s_step) : 0u), live ? s_bytes : 0u);
    dma4(lds_s + (uint32_t)(s & 3) * kScaleSlot, s_voff, r);
  };
  auto issue_middle = [&](int s) {   // what the middle of step s - 2 frees
    issue_w(s);
    issue_x(s, 0);
    issue_s(s);
  };

  // ---- fragments: line base + 16 f + i, pieces g and 4 + g (the codes 16 g .. and 64 + 16 g .. of the block)
  const uint32_t frag = (uint32_t)i * kB + (uint32_t)((g ^ (i >> 1)) << 4);
  const uint32_t rx = (uint32_t)(128 * gp) * kB + frag, rw = kSide + (uint32_t)(64 * wq) * kB + frag;
  const uint32_t rsx = kOffScale + 4u * (uint32_t)(128 * gp + i);
  const uint32_t rsw = kOffScale + 4u * (uint32_t)(kTile + 64 * wq + (WLINE ? 4 * g : 0));
  auto fragment = [&](uint32_t at, int f) {
    const v4i lo = lds16(at, 2048 * f), hi = lds16(at ^ 64u, 2048 * f);
    return __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
  };

  v4f acc[8][4];
#pragma unroll
  for (int f = 0; f < 8; ++f)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[f][j] = {0.0f, 0.0f, 0.0f, 0.0f};

  issue_middle(0);
  issue_x(0, 1);
  issue_middle(1);
  issue_x(1, 1);
  wait_vm<11>();
  lds_barrier();
  for (int s = 0; s < nb; ++s) {
    const uint32_t so = (uint32_t)(s & 1) * kStage, ss = (uint32_t)(s & 3) * kScaleSlot;
    // W, the first half of X and the scales of step s: all but the second half of X of this step, and the
    // next step's nine
    v8i w[4];
    Wide ww[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      w[j] = fragment(rw + so, j);
      if (EXACT) ww[j] = widen<FW>(w[j]);
    }
    float sw1 = 0.0f;
    if (!WLINE) sw1 = *reinterpret_cast<const float*>(smem + rsw + ss);
    auto half_step = [&](int h) {
#pragma unroll
      for (int f = 4 * h; f < 4 * h + 4; ++f) {
        const v8i x = fragment(rx + so, f);
        const float sx = *reinterpret_cast<const float*>(smem + rsx + ss + 64 * f);
        v4f d[4];
        if (EXACT) {
          // the four chains of four in turn: an instruction never waits for the one before it
          const Wide xw = widen<FX>(x);
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
          for (int q = 0; q < 4; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) d[j] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(ww[j].p[q], xw.p[q], d[j], 0, 0, 0);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j) d[j] = block_fp8<FX, FW>(w[j], x);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          if (WLINE) {
            const v4f sw = *reinterpret_cast<const v4f*>(smem + rsw + ss + 64 * j);
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[f][j][r] = __builtin_fmaf(d[j][r], sx * sw[r], acc[f][j][r]);
          } else {
            const float sc = sx * sw1;
#pragma unroll
            for (int r = 0; r < 4; ++r) acc[f][j][r] = __builtin_fmaf(d[j][r], sc, acc[f][j][r]);
          }
        }
        // the sums of this X fragment are added here and now: the compiler would keep them, in registers that
        // there are not, past the middle of the step
        if (EXACT) {
          pin(acc[f]);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    };
    half_step(0);
    // (as in the exact kernels: without this the sums of the first half wait, multiplied twice each, in registers that
    // spill; 4096 x 4096 x 4096 137 us, with it 76; with W's tiles they fit, and 120 us become 125)
    if (WLINE && !EXACT) {
#pragma unroll
      for (int f = 0; f < 4; ++f) pin(acc[f]);
    }
    // the second half of X of this step: all but the next step's nine
    wait_vm<9>();
    lds_barrier();
    issue_middle(s + 2);
    half_step(1);
    wait_vm<9>();
    lds_barrier();
    issue_x(s + 2, 1);
  }
  // the epilogue writes where the loads of steps past the end (zeros) may still land
  wait_vm<0>();
  lds_barrier();

  epilogue<8, 4, kWaveOut>(a, t, acc, wid, lane, 128 * gp, 64 * wq);
}

template <int FX, int FW, bool EXACT, bool WLINE>
hipError_t launch_t(const GemmB128& a, hipStream_t stream) {
  static bool set[64] = {false};
  auto kern = k_gemm_b128<FX, FW, EXACT, WLINE>;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!set[dev]) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, kLds);
    if (e != hipSuccess) return e;
    set[dev] = true;
  }
  const Grid grid = grid_of(gemm_b128_tiles(a, kTile, kTile));
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(kThreads), kLds, stream, a);
  return hipGetLastError();
}

template <int FX, int FW>
hipError_t launch_f(const GemmB128& a, hipStream_t s) {
  if (a.exact) return a.w_line ? launch_t<FX, FW, true, true>(a, s) : launch_t<FX, FW, true, false>(a, s);
  return a.w_line ? launch_t<FX, FW, false, true>(a, s) : launch_t<FX, FW, false, false>(a, s);
}

}  // namespace

hipError_t launch_gemm_b128_tile(const GemmB128& a, hipStream_t s) {
  if (a.x_fmt == kE4M3) return a.w_fmt == kE4M3 ? launch_f<0, 0>(a, s) : launch_f<0, 1>(a, s);
  return a.w_fmt == kE4M3 ? launch_f<1, 0>(a, s) : launch_f<1, 1>(a, s);
}

}  // namespace mxq
