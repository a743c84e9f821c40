// gemm_fp4.hip -- Y = act(alpha * (X W) + bias) with W in MXFP4 and X in bf16 or MXFP4, for
// gfx950.  Exact products, FP32 sums (see fp4_mma.hpp).
#include "fp4_mma.hpp"

namespace mxq {
namespace {

constexpr int kWaves = 8;
constexpr int kThreads = 64 * kWaves;

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

// A workgroup computes 16 * MT rows x 16 * NT columns of Y, its eight waves taking the units
// of K in turn; their sums meet in LDS and are added in wave order.  Consecutive workgroups
// of an XCD take the row tiles of one column tile, which read the same part of W.
template <int XT, int MT, int NT, int D>
__global__ __launch_bounds__(kThreads) void k_gemm4_rows(const Fp4Args a, const GemmEpilogue ep) {
  extern __shared__ __align__(16) float part[];
  const int t = xcd_order(blockIdx.x, a.tiles_m * a.tiles_n);
  const int m0 = (t % a.tiles_m) * 16 * MT, n0 = (t / a.tiles_m) * 16 * NT;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  Rows<MT, NT> r;
  r.w = a.w + (int64_t)n0 * a.ld_w;
  r.ws = a.ws + (int64_t)n0 * a.ld_ws;
#pragma unroll
  for (int n = 0; n < NT; ++n) {                       // rows past the end read the last one again
    const int row = min(16 * n + i, a.N - 1 - n0);
    r.wo[n] = (uint32_t)(row * a.ld_w) + 16u * g;
    r.so[n] = (uint32_t)(row * a.ld_ws) + (uint32_t)g;
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    const int64_t row = min(m0 + 16 * m + i, a.M - 1);
    r.x[m] = a.x + row * a.ld_x;
    r.xs[m] = XT == kXFp4 ? a.xs + row * a.ld_xs : nullptr;
  }
  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = {0.0f, 0.0f, 0.0f, 0.0f};
  sum_units<XT, MT, NT, D>(r, wave, kWaves, g, a.K, acc);
  store_part<MT, NT>(part, wave, lane, acc);
  __syncthreads();
  for (int q = threadIdx.x; q < 16 * MT * 4 * NT; q += kThreads) {
    const int m = q / (4 * NT), n = 4 * (q % (4 * NT));
    if (m0 + m < a.M && n0 + n < a.N)
      store4(ep, m0 + m, n0 + n, a.N, sum_part<MT, NT>(part, kWaves, m, n));
  }
}

template <int XT, int MT, int NT, int D>
hipError_t launch_rows(Fp4Args a, const GemmEpilogue& ep, hipStream_t st) {
  a.tiles_m = (a.M + 16 * MT - 1) / (16 * MT);
  a.tiles_n = (a.N + 16 * NT - 1) / (16 * NT);
  if ((int64_t)a.tiles_m * a.tiles_n > 0x7FFFFFFF) return hipErrorInvalidValue;
  constexpr int lds = kWaves * part_wave<MT, NT>() * 4;
  auto kern = k_gemm4_rows<XT, MT, NT, D>;
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
  hipLaunchKernelGGL(kern, dim3((unsigned)(a.tiles_m * a.tiles_n)), dim3(kThreads), lds, st, a, ep);
  return hipGetLastError();
}

// Columns per workgroup: as many as still give every CU a workgroup.
template <int XT, int MT>
hipError_t launch_m(const Fp4Args& a, const GemmEpilogue& ep, hipStream_t st) {
  const int64_t tm = (a.M + 16 * MT - 1) / (16 * MT);
  const int64_t cus = device_cu_count();
  if (tm * ((a.N + 63) / 64) >= cus) return launch_rows<XT, MT, 4, 2>(a, ep, st);
  if (tm * ((a.N + 31) / 32) >= cus) return launch_rows<XT, MT, 2, 2>(a, ep, st);
  return launch_rows<XT, MT, 1, MT == 1 ? 4 : 2>(a, ep, st);
}

template <int XT>
hipError_t launch_x(const Fp4Args& a, const GemmEpilogue& ep, hipStream_t st) {
  if (a.M <= 16) return launch_m<XT, 1>(a, ep, st);
  if (a.M <= 32) return launch_m<XT, 2>(a, ep, st);
  return launch_m<XT, 4>(a, ep, st);
}

}  // namespace

hipError_t launch_gemm_fp4(int64_t M, int64_t N, int64_t K, const void* x, bool x_fp4, int64_t ld_x, const uint8_t* xs,
                           int64_t ld_xs, const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws,
                           const GemmEpilogue& ep, hipStream_t st) {
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
  return x_fp4 ? launch_x<kXFp4>(a, ep, st) : launch_x<kXBf16>(a, ep, st);
}

}  // namespace mxq
