// gemm_fp4.hip -- Y = act(alpha * (X W) + bias) with W in MXFP4 and X in bf16 or MXFP4, for
// gfx950: the choice of kernel, and the kernel of few rows or tiles (fp4_stream.hpp).
#include "fp4_stream.hpp"

namespace mxq {
namespace {

struct Fp4Args {
  int M, N, K, tiles_m, tiles_n;
  const uint8_t* x;
  int64_t ld_x;                        // bytes
  const uint8_t* xs;
  int64_t ld_xs;
  const uint8_t* w;
  int64_t ld_w;
  const uint8_t* ws;
  int64_t ld_ws;
  bool x_pieces;                       // X rows are whole 16-byte pieces
  bool xs_words, ws_words;             // scale rows are whole 4-byte words
};

__device__ __forceinline__ void store4(const GemmEpilogue& ep, int64_t row, int col, int N, v4f v) {
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    const float b = ep.bias && col + e < N ? ep.bias[col + e] : -0.0f;
    v[e] = __builtin_fmaf(ep.alpha, v[e], b);
    if (ep.act) v[e] = silu(v[e]);
  }
  if (ep.y_bf16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(ep.y) + row * ep.ld_y + col;
    const uint32_t d[2] = {pack_bf16(v[0], v[1]), pack_bf16(v[2], v[3])};
    if (col + 4 <= N) {
      __builtin_memcpy(p, d, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < N) p[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* p = reinterpret_cast<float*>(ep.y) + row * ep.ld_y + col;
    if (col + 4 <= N) {
      __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < N) p[e] = v[e];
    }
  }
}

// A workgroup computes 16 * MT rows x 16 * NTW columns of Y.  Consecutive workgroups of an XCD
// take the row tiles of one column tile, which read the same part of W.
// How X comes: in MXFP4 through the ring, in bf16 staged by DMA or through registers.
enum : int { kFp4Ring = 0, kBf16Dma = 1, kBf16Regs = 2 };

template <int WAY, int MT, int NTW>
__global__ __launch_bounds__(kThreads, WAY == kFp4Ring ? 2 : 1) void k_gemm4_stream(const Fp4Args a, const GemmEpilogue ep) {
  const int wg = xcd_order(blockIdx.x, a.tiles_m * a.tiles_n);
  const int m0 = (wg % a.tiles_m) * 16 * MT, n0 = (wg / a.tiles_m) * 16 * NTW;
  const int lane = threadIdx.x & 63, i = lane & 15;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nb = (a.K + 31) / 32;
  const Lines w = lines_of(a.w + n0 * a.ld_w, a.ld_w, a.ws + n0 * a.ld_ws, a.ld_ws, min(16 * NTW, a.N - n0), nb, a.ws_words);
  const ItemOffsets wo = item_offsets(w.ld_c, w.ld_s, lane);
  auto issue = [&](int t, int c, uint32_t lds) { issue_item(w, wo, t, c, lds); };
  auto scales_of = [&](int t, int c, uint32_t slot) { return item_scales(w, slot, t, c, nb, lane); };
  const uint32_t ring = (uint32_t)wave * kWaveLds, lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem + ring;
  v4f acc[MT][NTW];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NTW; ++n) acc[m][n] = {0.0f, 0.0f, 0.0f, 0.0f};
  const Run run = run_of<NTW>(a.K, wave);
  if constexpr (WAY == kFp4Ring) {
    const Lines xl = lines_of(a.x + m0 * a.ld_x, a.ld_x, a.xs + m0 * a.ld_xs, a.ld_xs, min(16 * MT, a.M - m0), nb, a.xs_words);
    const ItemOffsets xo = item_offsets(xl.ld_c, xl.ld_s, lane);
    stream<XFp4<MT>, MT, NTW>(run, wave, lane, a.ws_words, false, issue, [&](XFp4<MT>& x, int c) {
      static_assert(MT <= kRing, "X tiles pass through the ring");
#pragma unroll
      for (int m = 0; m < MT; ++m) issue_item(xl, xo, m, c, lds0 + m * kSlot);
      wait_vm<0>();
      asm volatile("" ::: "memory");
#pragma unroll
      for (int m = 0; m < MT; ++m) {
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          x.f[u][m] = item_codes(ring + m * kSlot, lane, u);
          if (kChunk * (c + 1) > a.K) x.f[u][m] = keep_codes(x.f[u][m], a.K - kChunk * c - 32 * (4 * (lane >> 4) + u));
        }
        x.s[m] = item_scales(xl, ring + m * kSlot, m, c, nb, lane);
      }
      reads_done();
    }, scales_of, acc);
  } else {
    XStage<WAY == kBf16Dma, MT> xs;
#pragma unroll
    for (int m = 0; m < MT; ++m) xs.row[m] = a.x + min((int64_t)m0 + 16 * m + i, (int64_t)a.M - 1) * a.ld_x;
    xs.K = a.K;
    xs.lane = lane;
    xs.at = (uint32_t)wave * kStagedLds + kWaveLds;
    stream_staged<WAY == kBf16Dma, MT, NTW>(run, wave, lane, xs, issue, scales_of, acc);
  }
  __syncthreads();
  store_part<MT, NTW>(wave, lane, acc);
  __syncthreads();
  for (int q = threadIdx.x; q < 16 * MT * 4 * NTW; q += kThreads) {
    const int m = q / (4 * NTW), n = 4 * (q % (4 * NTW));
    if (m0 + m < a.M && n0 + n < a.N) store4(ep, m0 + m, n0 + n, a.N, sum_part<MT, NTW>(m, n));
  }
}

template <int WAY, int MT, int NTW>
hipError_t launch_stream(Fp4Args a, const GemmEpilogue& ep, hipStream_t st) {
  static bool set[64] = {false};
  a.tiles_m = (a.M + 16 * MT - 1) / (16 * MT);
  a.tiles_n = (a.N + 16 * NTW - 1) / (16 * NTW);
  if ((int64_t)a.tiles_m * a.tiles_n > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = k_gemm4_stream<WAY, MT, NTW>;
  constexpr int lds = stream_lds<MT, NTW, WAY == kFp4Ring ? kWaveLds : kStagedLds>();
  const hipError_t e = allow_lds(kern, lds, set);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(kThreads), lds, st, a, ep);
  return hipGetLastError();
}

// Columns per workgroup: as many as still give every CU a workgroup.
template <int WAY, int MT>
hipError_t launch_m(const Fp4Args& a, const GemmEpilogue& ep, hipStream_t st) {
  const int64_t tm = (a.M + 16 * MT - 1) / (16 * MT);
  const int64_t cus = device_cu_count();
  if constexpr (MT == 1 && WAY == kFp4Ring)
    if (tm * ((a.N + 127) / 128) >= cus) return launch_stream<WAY, MT, 8>(a, ep, st);
  if (tm * ((a.N + 63) / 64) >= cus) return launch_stream<WAY, MT, 4>(a, ep, st);
  if (tm * ((a.N + 31) / 32) >= cus) return launch_stream<WAY, MT, 2>(a, ep, st);
  return launch_stream<WAY, MT, 1>(a, ep, st);
}

}  // namespace

hipError_t launch_gemm_fp4(int64_t M, int64_t N, int64_t K, const void* x, bool x_fp4, int64_t ld_x, const uint8_t* xs,
                           int64_t ld_xs, const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws,
                           const GemmEpilogue& ep, hipStream_t st) {
  auto whole = [](const void* p, int64_t ld, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0 && ld % n == 0; };
  // 256 x 256 tiles once they fill half the CUs: 2048 x 4096 x 4096 takes 31 us so and 47 as a stream,
  // 1024 x 4096 x 4096 (64 tiles) 30 and 23
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  if (x_fp4 && K > 0 && 2 * tiles >= device_cu_count() && whole(xs, ld_xs, 16) && whole(ws, ld_ws, 16))
    return launch_gemm_fp4_tile(M, N, K, (const uint8_t*)x, ld_x, xs, ld_xs, wc, ld_w, ws, ld_ws, ep, st);
  Fp4Args a{};
  a.M = (int)M;
  a.N = (int)N;
  a.K = (int)K;
  a.x = (const uint8_t*)x;
  a.ld_x = x_fp4 ? ld_x : 2 * ld_x;
  a.xs = xs;
  a.ld_xs = ld_xs;
  a.w = wc;
  a.ld_w = ld_w;
  a.ws = ws;
  a.ld_ws = ld_ws;
  a.x_pieces = whole(x, a.ld_x, 16);
  a.xs_words = whole(xs, ld_xs, 4);
  a.ws_words = whole(ws, ld_ws, 4);
  if (x_fp4) {
    if (M <= 16) return launch_m<kFp4Ring, 1>(a, ep, st);
    return M <= 32 ? launch_m<kFp4Ring, 2>(a, ep, st) : launch_m<kFp4Ring, 4>(a, ep, st);
  }
  // whole 16-byte pieces, the last one of a row included, and scales in whole words
  if (a.x_pieces && K % 8 == 0 && a.ws_words) return M <= 16 ? launch_m<kBf16Dma, 1>(a, ep, st) : launch_m<kBf16Dma, 2>(a, ep, st);
  return M <= 16 ? launch_m<kBf16Regs, 1>(a, ep, st) : launch_m<kBf16Regs, 2>(a, ep, st);
}

}  // namespace mxq
