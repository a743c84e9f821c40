// gemm_b128_rows.hip -- the product in blocks of 128 by small tiles whose eight waves split K: few rows (a
// decoding step, a few tokens an expert), and outputs too small to fill the card with 256 x 256 tiles.
//
// Bound by the weights' bytes and by latency.  A workgroup owns 16 MT x 16 NT outputs; wave v takes blocks v,
// v + 8, ..., so that the eight together read 1 KiB runs of each line.  Codes come straight from memory into
// the fragments' registers, U blocks at a time and the next U on their way while these are multiplied; the
// eight waves' sums meet in LDS, are added in the waves' order, and finished by all threads.
#include "gemm_b128.hpp"

namespace mxq {
namespace {

constexpr int kThreads = 512;
constexpr int kWaves = 8;

template <int FX, int FW, bool EXACT, bool WLINE, int MT, int NT, int U>
struct RowsWave {
  struct Batch {
    v4i x[U][MT][2], w[U][NT][2];
    float sx[U][MT];
    v4f sw[U][WLINE ? NT : 1];
  };
  __amdgpu_buffer_rsrc_t rx, rw, rsx, rsw;
  uint32_t vx, vw;
  int64_t ld_xs, ws_k;
  uint32_t x16, w16;
  int nb, i, g;

  __device__ __forceinline__ void load(Batch& q, int b0) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + kWaves * u;
      const uint32_t dead = b < nb ? 0u : 0x80000000u;     // past every range (each below 2^31): loads give zeros
      const uint32_t at = (uint32_t)b * kB;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q.w[u][j][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rw, (int)((vw + j * w16 + 64 * h + at) | dead), 0, 0));
#pragma unroll
      for (int f = 0; f < MT; ++f)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          q.x[u][f][h] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(rx, (int)((vx + f * x16 + 64 * h + at) | dead), 0, 0));
      const uint32_t sa = (uint32_t)(4 * (b * ld_xs + i));
#pragma unroll
      for (int f = 0; f < MT; ++f)
        q.sx[u][f] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsx, (int)((sa + 64 * f) | dead), 0, 0));
      const uint32_t wa = (uint32_t)(4 * (b * ws_k + (WLINE ? 4 * g : 0)));
      if (WLINE) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
          q.sw[u][j] = __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(rsw, (int)((wa + 64 * j) | dead), 0, 0));
      } else {
        q.sw[u][0][0] = __uint_as_float(__builtin_amdgcn_raw_buffer_load_b32(rsw, (int)(wa | dead), 0, 0));
      }
    }
  }
  __device__ __forceinline__ void multiply(const Batch& q, v4f acc[MT][NT]) const {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      v8i w[NT];
      Wide ww[NT];
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        w[j] = __builtin_shufflevector(q.w[u][j][0], q.w[u][j][1], 0, 1, 2, 3, 4, 5, 6, 7);
        if (EXACT) ww[j] = widen<FW>(w[j]);
      }
#pragma unroll
      for (int f = 0; f < MT; ++f) {
        const v8i x = __builtin_shufflevector(q.x[u][f][0], q.x[u][f][1], 0, 1, 2, 3, 4, 5, 6, 7);
        Wide xw;
        if (EXACT) xw = widen<FX>(x);
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const v4f d = EXACT ? block_exact(ww[j], xw) : block_fp8<FX, FW>(w[j], x);
#pragma unroll
          for (int r = 0; r < 4; ++r)
            acc[f][j][r] = __builtin_fmaf(d[r], q.sx[u][f] * (WLINE ? q.sw[u][j][r] : q.sw[u][0][0]), acc[f][j][r]);
        }
      }
    }
  }
};

template <int FX, int FW, bool EXACT, bool WLINE, int MT, int NT>
__global__ __launch_bounds__(kThreads, 2) void k_gemm_b128_rows(const GemmB128 a) {
  constexpr int U = MT + NT <= 2 ? 4 : MT + NT <= 4 ? 2 : 1;
  const B128Tile t = b128_tile<16 * MT, 16 * NT, WLINE>(a, workgroup_at(blockIdx.x, blockIdx.y));
  if (!t.any) return;
  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int rows_x = min(16 * MT, t.m), rows_w = min(16 * NT, t.n);
  using Wave = RowsWave<FX, FW, EXACT, WLINE, MT, NT, U>;
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
  typename Wave::Batch p, q;
  constexpr int step = kWaves * U;
  v.load(p, wid);
  for (int b = wid; b < t.nb; b += 2 * step) {
    v.load(q, b + step);
    v.multiply(p, acc);
    v.load(p, b + 2 * step);
    v.multiply(q, acc);
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
    for (int w = 1; w < kWaves; ++w) {
      const v4f e = part[w * MT * NT * 64 + o];
#pragma unroll
      for (int r = 0; r < 4; ++r) s[r] += e[r];
    }
    const int l = o & 63, f = (o >> 6) / NT, j = (o >> 6) % NT;
    const int m = 16 * f + (l & 15), n = 16 * j + 4 * (l >> 4);
    if (m >= rows_x || n >= rows_w) continue;
    const int left = rows_w - n;
#pragma unroll
    for (int r = 0; r < 4; ++r)
      s[r] = finish(s[r], a.alpha, a.bias && r < left ? a.bias[t.n0 + n + r] : -0.0f, a.act);
    const int64_t at = t.y + (int64_t)m * a.ld_y + n;
    if (a.y_bf16) {
      uint16_t* y = reinterpret_cast<uint16_t*>(a.y) + at;
      const v2u d = {pack_bf16(s[0], s[1]), pack_bf16(s[2], s[3])};
      if (a.y_vec16 && left >= 4) {
        *reinterpret_cast<v2u*>(y) = d;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r < left) y[r] = (uint16_t)(d[r >> 1] >> (16 * (r & 1)));
      }
    } else {
      float* y = reinterpret_cast<float*>(a.y) + at;
      if (a.y_vec16 && left >= 4) {
        *reinterpret_cast<v4f*>(y) = s;
      } else {
#pragma unroll
        for (int r = 0; r < 4; ++r)
          if (r < left) y[r] = s[r];
      }
    }
  }
}

template <int FX, int FW, bool EXACT, bool WLINE, int MT, int NT>
hipError_t launch_t(const GemmB128& a, hipStream_t stream) {
  constexpr int lds = kWaves * MT * NT * 1024;
  auto kern = k_gemm_b128_rows<FX, FW, EXACT, WLINE, MT, NT>;
  if (lds > 65536) {
    static bool set[64] = {false};
    int dev = 0;
    if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
    if (!set[dev]) {
      const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, lds);
      if (e != hipSuccess) return e;
      set[dev] = true;
    }
  }
  const Grid grid = grid_of(gemm_b128_tiles(a, 16 * MT, 16 * NT));
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(kThreads), lds, stream, a);
  return hipGetLastError();
}

template <int FX, int FW, bool EXACT, bool WLINE>
hipError_t launch_p(const GemmB128& a, const GemmB128Plan& p, hipStream_t s) {
  if (p.tile_m == 16) return p.tile_n == 16 ? launch_t<FX, FW, EXACT, WLINE, 1, 1>(a, s) : launch_t<FX, FW, EXACT, WLINE, 1, 2>(a, s);
  if (p.tile_m == 32) return p.tile_n == 16 ? launch_t<FX, FW, EXACT, WLINE, 2, 1>(a, s) : launch_t<FX, FW, EXACT, WLINE, 2, 2>(a, s);
  return p.tile_n == 32 ? launch_t<FX, FW, EXACT, WLINE, 4, 2>(a, s) : launch_t<FX, FW, EXACT, WLINE, 4, 4>(a, s);
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
