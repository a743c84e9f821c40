// gemm_fp4.hip -- Y = act(alpha * (X W) + bias) with W in MXFP4 and X in bf16 or MXFP4, for
// gfx950: the choice of kernel, the kernel of few rows or tiles, and the one of K < 8.  The large product of two
// MXFP4 operands is in gemm_fp4_tile.hip.
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
    if (whole_group(col, N)) {
      __builtin_memcpy(p, d, 8);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < N) p[e] = (uint16_t)(d[e >> 1] >> (16 * (e & 1)));
    }
  } else {
    float* p = reinterpret_cast<float*>(ep.y) + row * ep.ld_y + col;
    if (whole_group(col, N)) {
      __builtin_memcpy(p, &v, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e)
        if (col + e < N) p[e] = v[e];
    }
  }
}

// A workgroup computes a tile of 16 * MT rows x 16 * NT columns of Y; its waves (1 to 8) split K in
// runs of whole kRun elements, and their sums meet in LDS, added in wave order.  A wave has its
// piece of both operands to itself: rows are loaded whole lines at a time into registers (8 lanes
// a row; any alignment of X in bf16 and of the scales), put into the wave's own LDS, swizzled, and
// read back as fragments, so there is no barrier before the sums and the next piece is on its way
// while one is multiplied.
// LDS is written and read in different types.
typedef uint16_t u16a __attribute__((may_alias));
typedef uint32_t u32a __attribute__((may_alias));
typedef uint64_t u64a __attribute__((may_alias));

constexpr int kRun = 128;              // granularity of a wave's share of K
constexpr int kPiece = 256;            // elements of K of an MXFP4 operand per load
constexpr int kUnit = 64;              // and of X in bf16

// LDS of one piece of 16 * T rows: codes (128 bytes a row, 16-byte block p of row r at p ^ (r & 7))
// and 8 scale bytes a row.
constexpr int rows4_lds(int t) { return t * (2048 + 128); }

// 16 * T rows of MXFP4.
template <int T>
struct Rows4 {
  __amdgpu_buffer_rsrc_t codes;
  uint32_t off[2 * T];                 // rows 8d + (lane >> 3), block lane & 7
  const uint8_t* scales;               // the lane's row (lanes past 16 * T repeat the last one)
  int K, nb, lane;

  struct Raw {
    v4i c[2 * T];
    uint64_t s;
  };

  // Rows `row0` .. of `rows`: those past the end are read as the last one.
  __device__ __forceinline__ void init(const uint8_t* c, int64_t ld_c, const uint8_t* s, int64_t ld_s, int64_t row0, int rows,
                                       int k, int ln) {
    K = k;
    nb = (k + 31) / 32;
    lane = ln;
    const int last = min(16 * T, (int)(rows - row0)) - 1;
    codes = make_rsrc(c + row0 * ld_c, (uint32_t)((int64_t)last * ld_c + 16 * nb));
#pragma unroll
    for (int d = 0; d < 2 * T; ++d) off[d] = (uint32_t)min(8 * d + (lane >> 3), last) * (uint32_t)ld_c + 16u * (lane & 7);
    scales = s + (row0 + min(lane, last)) * ld_s;
  }

  // Elements k0 .. of the rows, those before `end` (both whole blocks; no load goes past the
  // last block).
  __device__ __forceinline__ void ask(Raw& r, int k0, int end) const {
    const int b0 = k0 / 32;
    const bool in = 32 * (b0 + (lane & 7)) < end && b0 + (lane & 7) < nb;
#pragma unroll
    for (int d = 0; d < 2 * T; ++d)
      r.c[d] = __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(codes, in ? (int)(off[d] + 16u * b0) : -16, 0, 0));
    r.s = 0;
    if (nb >= 8) {                     // the last 8 bytes of a row serve a piece that is cut
      __builtin_memcpy(&r.s, scales + min(b0, nb - 8), 8);
    } else {
#pragma unroll 1
      for (int b = 0; b < nb; ++b) r.s |= (uint64_t)scales[b] << (8 * b);
    }
  }

  // Into LDS.  Elements past K become code 0, blocks past it scale 1.
  __device__ __forceinline__ void put(Raw& r, int k0, uint32_t lds) const {
    const int b0 = k0 / 32;
    if (k0 + kPiece > K) {
      const v4i keep = keep_codes(v4i{-1, -1, -1, -1}, K - k0 - 32 * (lane & 7));
#pragma unroll
      for (int d = 0; d < 2 * T; ++d) r.c[d] &= keep;
      r.s >>= 8 * (b0 - max(min(b0, nb - 8), 0));
      const int left = nb - b0;        // 1 .. 8
      if (left < 8) {
        const uint64_t m = ~0ull << (8 * left);
        r.s = (r.s & ~m) | (0x7F7F7F7F7F7F7F7Full & m);
      }
    }
#pragma unroll
    for (int d = 0; d < 2 * T; ++d)
      *reinterpret_cast<v4i*>(smem + lds + 1024 * d + 128 * (lane >> 3) + 16 * ((lane & 7) ^ (lane >> 3))) = r.c[d];
    if (lane < 16 * T) *reinterpret_cast<u64a*>(smem + lds + 2048 * T + 8 * lane) = r.s;
  }
};

// Eight 16-bit elements without the first n (0 .. 8), zeros behind.
__device__ __forceinline__ v4i without_first(v4i v, int n) {
  uint64_t lo = (uint32_t)v[0] | ((uint64_t)(uint32_t)v[1] << 32), hi = (uint32_t)v[2] | ((uint64_t)(uint32_t)v[3] << 32);
  if (n >= 4) {
    lo = n == 8 ? 0 : hi;
    hi = 0;
  }
  const int s = 16 * (n & 3);
  lo = (lo >> s) | (hi << 1 << (63 - s));
  hi >>= s;
  return v4i{(int)lo, (int)(lo >> 32), (int)hi, (int)(hi >> 32)};
}

// 16 * T rows of bf16, kUnit elements at a time: the same lines of 128 bytes.
template <int T>
struct RowsBf16 {
  const uint8_t* row[2 * T];
  int K, lane;

  struct Raw {
    v4i v[2 * T];
  };

  __device__ __forceinline__ void init(const uint8_t* x, int64_t ld, int64_t row0, int rows, int k, int ln) {
    K = k;
    lane = ln;
#pragma unroll
    for (int d = 0; d < 2 * T; ++d) row[d] = x + min(row0 + 8 * d + (lane >> 3), (int64_t)rows - 1) * ld;
  }

  // Elements k0 + 8 * (lane & 7) ..; the piece that the row's end cuts, and those past it, are read
  // from its last 8 elements (K >= 8).
  __device__ __forceinline__ void ask(Raw& r, int k0) const {
    const int64_t at = 2 * (int64_t)min(k0 + 8 * (lane & 7), K - 8);
#pragma unroll
    for (int d = 0; d < 2 * T; ++d) __builtin_memcpy(&r.v[d], row[d] + at, 16);
  }

  __device__ __forceinline__ void put(Raw& r, int k0, uint32_t lds) const {
    if (k0 + kUnit > K) {
      const int cut = min(max(k0 + 8 * (lane & 7) + 8 - K, 0), 8);
#pragma unroll
      for (int d = 0; d < 2 * T; ++d) r.v[d] = without_first(r.v[d], cut);
    }
#pragma unroll
    for (int d = 0; d < 2 * T; ++d)
      *reinterpret_cast<v4i*>(smem + lds + 1024 * d + 128 * (lane >> 3) + 16 * ((lane & 7) ^ (lane >> 3))) = r.v[d];
  }
};

constexpr int split_row(int nt) { return 16 * nt + 4; }   // floats of a row of a wave's sums
constexpr int split_wave_lds(bool x_fp4, int mt, int nt) { return rows4_lds(nt) + (x_fp4 ? rows4_lds(mt) : 2048 * mt); }
constexpr int split_lds(bool x_fp4, int split, int mt, int nt) {
  const int stage = split * split_wave_lds(x_fp4, mt, nt), sums = split * 16 * mt * split_row(nt) * 4;
  return stage > sums ? stage : sums;
}

// X in MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4, lane (i, g) holding block 4v + g of row i.
template <int MT, int NT>
__device__ __forceinline__ void multiply_fp4(uint32_t w, uint32_t x, int lane, v4f acc[MT][NT]) {
  const uint32_t i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int v = 0; v < 2; ++v) {
    v4i xf[MT];
    uint32_t xs[MT];
    const uint32_t at = 128 * i + 16 * ((4 * v + g) ^ (i & 7));
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      xf[m] = lds16(x + at, 2048 * m);
      xs[m] = smem[x + 2048 * MT + 8 * i + 4 * v + g + 128 * m];
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const v4i wf = lds16(w + at, 2048 * n);
      const uint32_t ws = smem[w + 2048 * NT + 8 * i + 4 * v + g + 128 * n];
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][n] = mma_fp4<0>(wf, ws, xf[m], xs[m], acc[m][n]);
    }
  }
}

// Unit u of a piece of W with X in bf16: lane (i, g) holds elements 8g .. 8g+7 of both blocks of
// row i, W decoded with its scale (exact).
template <int MT, int NT>
__device__ __forceinline__ void multiply_bf16(uint32_t w, uint32_t x, int u, int lane, v4f acc[MT][NT]) {
  const uint32_t i = lane & 15, g = lane >> 4;
  v4i xf[MT][2];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int j = 0; j < 2; ++j) xf[m][j] = lds16(x + 128 * i + 16 * ((g + 4 * j) ^ (i & 7)), 2048 * m);
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint32_t s = *reinterpret_cast<const u16a*>(smem + w + 2048 * NT + 128 * n + 8 * i + 2 * u);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t d[4];
      fp4::decode8_bf16(*reinterpret_cast<const u32a*>(smem + w + 2048 * n + 128 * i + 16 * ((2 * u + j) ^ (i & 7)) + 4 * g),
                        e8m0_to_f32(j ? s >> 8 : s & 255u), d);
      const v4i wf = {(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
#pragma unroll
      for (int m = 0; m < MT; ++m) acc[m][n] = mma_bf16(wf, xf[m][j], acc[m][n]);
    }
  }
}

template <bool X_FP4, int SPLIT, int MT, int NT>
__global__ __launch_bounds__(64 * SPLIT, 2) void k_gemm4_split(const Fp4Args a, const GemmEpilogue ep) {
  // in groups of four tile rows, so that what an XCD works on at a time shares rows of both operands: column
  // by column over all rows 8192 x 4096 x 4096 with X in bf16 took 565 us against 315, 8192 x 500 x 1500 in
  // MXFP4 19.4 against 13.9
  const int wg = workgroup_at(blockIdx.x, blockIdx.y);
  if (blockIdx.y > 0 && wg >= a.tiles_m * a.tiles_n) return;
  int tm, tn;
  tile_of(wg, a.tiles_m, a.tiles_n, tm, tn);
  const int m0 = tm * 16 * MT, n0 = tn * 16 * NT;
  const int lane = threadIdx.x & 63, i = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const uint32_t lw = (uint32_t)wave * split_wave_lds(X_FP4, MT, NT), lx = lw + rows4_lds(NT);
  const int runs = (a.K + kRun - 1) / kRun;
  const int k1 = min((int)((int64_t)runs * (wave + 1) / SPLIT) * kRun, a.K);
  int k = (int)((int64_t)runs * wave / SPLIT) * kRun;
  v4f acc[MT][NT];
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n] = {0.0f, 0.0f, 0.0f, 0.0f};
  Rows4<NT> w;
  w.init(a.w, a.ld_w, a.ws, a.ld_ws, n0, a.N, a.K, lane);
  typename Rows4<NT>::Raw rw;
  if constexpr (X_FP4) {
    Rows4<MT> x;
    x.init(a.x, a.ld_x, a.xs, a.ld_xs, m0, a.M, a.K, lane);
    typename Rows4<MT>::Raw rx;
    if (k < k1) {
      x.ask(rx, k, k1);
      w.ask(rw, k, k1);
    }
#pragma unroll 1
    for (; k < k1; k += kPiece) {
      x.put(rx, k, lx);
      w.put(rw, k, lw);
      if (k + kPiece < k1) {
        x.ask(rx, k + kPiece, k1);
        w.ask(rw, k + kPiece, k1);
      }
      multiply_fp4<MT, NT>(lw, lx, lane, acc);
    }
  } else {
    RowsBf16<MT> x;
    x.init(a.x, a.ld_x, m0, a.M, a.K, lane);
    typename RowsBf16<MT>::Raw rx;
    if (k < k1) {
      x.ask(rx, k);
      w.ask(rw, k, k1);
    }
    // one loop for all units: its instructions are fetched once
    int u = 0;
#pragma unroll 1
    for (; k < k1; k += kUnit) {
      if (u == 0) {
        w.put(rw, k, lw);
        if (k + kPiece < k1) w.ask(rw, k + kPiece, k1);
      }
      x.put(rx, k, lx);
      if (k + kUnit < k1) x.ask(rx, k + kUnit);
      multiply_bf16<MT, NT>(lw, lx, u, lane, acc);
      u = (u + 1) % (kPiece / kUnit);
    }
  }
  __syncthreads();
  float* part = reinterpret_cast<float*>(smem);
  constexpr int kRow = split_row(NT), kWave = 16 * MT * kRow;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) *reinterpret_cast<v4f*>(part + wave * kWave + (16 * m + i) * kRow + 16 * n + 4 * g) = acc[m][n];
  __syncthreads();
  for (int q = threadIdx.x; q < 16 * MT * 4 * NT; q += 64 * SPLIT) {
    const int m = q / (4 * NT), n = 4 * (q % (4 * NT));
    if (m0 + m >= a.M || n0 + n >= a.N) continue;
    v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int wv = 0; wv < SPLIT; ++wv) s += *reinterpret_cast<const v4f*>(part + wv * kWave + m * kRow + n);
    store4(ep, m0 + m, n0 + n, a.N, s);
  }
}

// K < 8 with X in bf16, where a row has no whole 16-byte piece: a thread four columns of a row of Y.
__global__ __launch_bounds__(256) void k_gemm4_short(const Fp4Args a, const GemmEpilogue ep) {
  const int n4 = column_groups(a.N);
  const int64_t q = workgroup_at(blockIdx.x, blockIdx.y) * 256ll + threadIdx.x;
  const int64_t m = q / n4;
  const int n0 = 4 * (int)(q % n4);
  if (m >= a.M) return;
  v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int e = 0; e < 4 && n0 + e < a.N; ++e) {
    const float scale = e8m0_to_f32(a.ws[(n0 + e) * a.ld_ws]);
    uint32_t c;
    __builtin_memcpy(&c, a.w + (n0 + e) * a.ld_w, 4);
    for (int k = 0; k < a.K; ++k) {
      float v[4];
      fp4::decode4_f32(c >> (4 * k), scale, v);
      s[e] += v[0] * __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(a.x + m * a.ld_x)[k] << 16);
    }
  }
  store4(ep, m, n0, a.N, s);
}

template <bool X_FP4, int SPLIT, int MT, int NT>
hipError_t launch_split(Fp4Args a, const GemmEpilogue& ep, hipStream_t st) {
  static bool set[64] = {false};
  a.tiles_m = (int)((a.M + 16ll * MT - 1) / (16 * MT));
  a.tiles_n = (int)((a.N + 16ll * NT - 1) / (16 * NT));
  if ((int64_t)a.tiles_m * a.tiles_n > 0x7FFFFFFF) return hipErrorInvalidValue;
  auto kern = k_gemm4_split<X_FP4, SPLIT, MT, NT>;
  constexpr int lds = split_lds(X_FP4, SPLIT, MT, NT);
  const hipError_t e = allow_lds(kern, lds, set);
  if (e != hipSuccess) return e;
  const Grid grid = grid_of((int64_t)a.tiles_m * a.tiles_n);
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(64 * SPLIT), lds, st, a, ep);
  return hipGetLastError();
}

// The tile and the split, from timing ten of them on 50 shapes (256 CUs).  Where 64 x 64 tiles fill the
// CUs, as many waves a tile as the card holds at once (8 a CU), up to 8: 1000 x 1000 x 4001 10.4 us with
// 8 (12.5 with 2), 2000 x 1000 x 3000 12.9 with 4 (14.8 with 2), 2048^3 14.1 with 2 (15.6 with 4), 3000 x 2500 x
// 2500 34.3 with 1 (36.1 with 4); with X in bf16 512 x 4096 x 4096 25 with 4 (35 with 2), 1024 rows 44 with 2 (46
// with 4), 2048 rows 81 with 1 (98 with 2).  K of at most 1024 leaves many waves less than a piece each: 64 x 32
// tiles by two waves for X in MXFP4 (3000 x 1500 x 800 12.8 us, 15.2 in 64 x 64 by four; 1500 x 4096 x 500
// 11.7 and 17.2), and 32 x 32 by four where there are fewer.  Else the largest tile that still gives
// every CU a workgroup, by four waves where it gives one to some CUs twice (30 x 32768 x 4096 20.7 us, 24.8
// by eight), and for up to 16 rows no wider than 32 columns (1 x 65536 x 4096 30.0 us, 46 with 64; 1 x 8192
// x 5120 7.1 and 11.3).
GemmFp4Plan rows_plan(int64_t M, int64_t N, int64_t K, bool x_fp4, int64_t cus) {
  auto tiles = [&](int mt, int nt) { return ((M + 16ll * mt - 1) / (16 * mt)) * ((N + 16ll * nt - 1) / (16 * nt)); };
  auto plan = [](int waves, int mt, int nt) { return GemmFp4Plan{16 * mt, 16 * nt, waves}; };
  const bool brief = K <= 1024;
  if (M > 32 && tiles(4, 4) > cus) {
    if (x_fp4 && brief) return plan(2, 4, 2);
    return plan(tiles(4, 4) <= 2 * cus ? 4 : tiles(4, 4) <= 4 * cus ? 2 : 1, 4, 4);
  }
  if (M > 32 && !brief && tiles(4, 4) == cus) return plan(8, 4, 4);
  if (M > 16) {
    if (brief && tiles(2, 2) >= cus) return plan(4, 2, 2);
    if (tiles(2, 4) > cus) return plan(4, 2, 4);
    if (tiles(2, 4) == cus) return plan(8, 2, 4);
    return plan(8, 2, tiles(2, 2) >= cus ? 2 : 1);
  }
  return plan(brief ? 4 : 8, 1, tiles(1, 2) >= cus ? 2 : 1);
}

template <bool X_FP4>
hipError_t launch_rows(const GemmFp4Plan& p, const Fp4Args& a, const GemmEpilogue& ep, hipStream_t st) {
  const int mt = p.tile_m / 16, nt = p.tile_n / 16;
  auto is = [&](int waves, int m, int n) { return p.waves == waves && mt == m && nt == n; };
  if constexpr (X_FP4) {
    if (is(2, 4, 2)) return launch_split<true, 2, 4, 2>(a, ep, st);
  }
  if (is(8, 4, 4)) return launch_split<X_FP4, 8, 4, 4>(a, ep, st);
  if (is(4, 4, 4)) return launch_split<X_FP4, 4, 4, 4>(a, ep, st);
  if (is(2, 4, 4)) return launch_split<X_FP4, 2, 4, 4>(a, ep, st);
  if (is(1, 4, 4)) return launch_split<X_FP4, 1, 4, 4>(a, ep, st);
  if (is(8, 2, 4)) return launch_split<X_FP4, 8, 2, 4>(a, ep, st);
  if (is(4, 2, 4)) return launch_split<X_FP4, 4, 2, 4>(a, ep, st);
  if (is(8, 2, 2)) return launch_split<X_FP4, 8, 2, 2>(a, ep, st);
  if (is(4, 2, 2)) return launch_split<X_FP4, 4, 2, 2>(a, ep, st);
  if (is(8, 2, 1)) return launch_split<X_FP4, 8, 2, 1>(a, ep, st);
  if (is(8, 1, 2)) return launch_split<X_FP4, 8, 1, 2>(a, ep, st);
  if (is(4, 1, 2)) return launch_split<X_FP4, 4, 1, 2>(a, ep, st);
  if (is(8, 1, 1)) return launch_split<X_FP4, 8, 1, 1>(a, ep, st);
  if (is(4, 1, 1)) return launch_split<X_FP4, 4, 1, 1>(a, ep, st);
  return hipErrorInvalidValue;
}

}  // namespace

GemmFp4Plan gemm_fp4_plan(int64_t M, int64_t N, int64_t K, bool x_fp4, bool aligned, int cus) {
  // 256 x 256 tiles from two for five CUs on: 4096 x 2048 x 4096 (128 tiles) takes 32 us so and 43 in small
  // tiles, 3000 x 2500 x 2500 (120) 28 and 34, 1500 x 4096 x 500 (96) 11.4 and 11.7, 1000 x 4096 x 4096 (64)
  // 30 and 24.  The tiles are counted, not how full they are: 30 x 32768 x 4096 (128) takes 29 us and would take
  // 13 in small ones.  The bias is read with 32-bit offsets.
  const int64_t tiles = ((M + 255) / 256) * ((N + 255) / 256);
  if (x_fp4 && K > 0 && 5 * tiles >= 2 * (int64_t)cus && N < (int64_t)1 << 29 && aligned) return GemmFp4Plan{256, 256, 8};
  if (!x_fp4 && K > 0 && K < 8) return GemmFp4Plan{1, 4, 0};
  return rows_plan(M, N, K, x_fp4, cus);
}

hipError_t launch_gemm_fp4(int64_t M, int64_t N, int64_t K, const void* x, bool x_fp4, int64_t ld_x, const uint8_t* xs,
                           int64_t ld_xs, const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws,
                           const GemmEpilogue& ep, hipStream_t st) {
  auto whole = [](const void* p, int64_t ld, int64_t n) { return (uintptr_t)p % (uintptr_t)n == 0 && ld % n == 0; };
  const GemmFp4Plan p = gemm_fp4_plan(M, N, K, x_fp4, whole(xs, ld_xs, 16) && whole(ws, ld_ws, 16), device_cu_count());
  if (p.tile_m == 256)
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
  if (p.waves == 0) {
    const int64_t blocks = (M * column_groups(a.N) + 255) / 256;
    if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
    const Grid grid = grid_of(blocks);
    hipLaunchKernelGGL(k_gemm4_short, dim3(grid.x, grid.y), dim3(256), 0, st, a, ep);
    return hipGetLastError();
  }
  return x_fp4 ? launch_rows<true>(p, a, ep, st) : launch_rows<false>(p, a, ep, st);
}

}  // namespace mxq
