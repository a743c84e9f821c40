// quantize_fp4.hip -- MXFP4 block quantization and dequantization for gfx950.
//
// Per 32-element block along K: amax, a power-of-two scale 2^e (the smallest with
// amax <= 6 * 2^e, or floor(log2 amax) - 2), the E8M0 byte e + 127 and 32 E2M1 codes of
// x / 2^e in 16 bytes (OCP Microscaling Formats Specification v1.0; the layout and scale
// policies are those of the 8-bit formats in quantize.hip).  2 or 4 bytes are read and 17/32 written
// per element and orientation.  HBM bounds rounding to nearest (8192 x 8192 bf16 along rows 37 us, 4.6
// TB/s, fp32 82 us, 3.7; 8192 x 4096 bf16 both ways 25 us, 4.1; dequantize 14 us, 6 TB/s, part of it from the
// last-level cache); stochastic rounding is bound
// by the integer multiplies of Philox, five of 32 x 32 bits an element (4096 x 4096 bf16 19 us
// along rows, 22 down columns; 4095 x 4001 fp32 down columns 25).
#include "codec4.hpp"
#include "fp4_ranges.hpp"
#include "internal.hpp"

namespace mxq {
namespace {

constexpr int kThreads = 256;
constexpr int kXcds = 8;
using namespace fp4;

// 16 bytes at any element alignment (one dwordx4 access; gfx950 takes unaligned addresses).
__device__ __forceinline__ uint4 load16(const void* p) {
  uint4 v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Elements k .. k+7 of a line whose valid elements are [0, K): those past the end read as zero.
template <int SRC_BF16>
__device__ __forceinline__ void load_chunk(Chunk<SRC_BF16>& c, const char* line, int64_t k, int64_t K) {
  constexpr int ES = SRC_BF16 ? 2 : 4;
  if (k + 8 <= K) {
#pragma unroll
    for (int h = 0; h < ES / 2; ++h) {
      const uint4 v = load16(line + k * ES + 16 * h);
      c.w[4 * h] = v.x;
      c.w[4 * h + 1] = v.y;
      c.w[4 * h + 2] = v.z;
      c.w[4 * h + 3] = v.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < (SRC_BF16 ? 4 : 8); ++i) {
      if (SRC_BF16) {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(line);
        const uint32_t lo = k + 2 * i < K ? p[k + 2 * i] : 0u;
        const uint32_t hi = k + 2 * i + 1 < K ? p[k + 2 * i + 1] : 0u;
        c.w[i] = lo | (hi << 16);
      } else {
        c.w[i] = k + i < K ? reinterpret_cast<const uint32_t*>(line)[k + i] : 0u;
      }
    }
  }
}

// Codes of a whole block, given as four chunks, under scale byte sb; stochastic when SR (the
// block's Philox words, block index in the padded code array).
template <int SRC_BF16, bool SR>
__device__ __forceinline__ uint4 encode32(const Chunk<SRC_BF16> c[4], uint32_t sb, uint64_t block, uint64_t seed) {
  uint32_t d[4];
  if (SR && sb != 255u) {
    uint32_t rnd[32];
    block_random(block, seed, rnd);
    const float inv = inv_scale_of(sb);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      d[q] = 0;
#pragma unroll
      for (int i = 0; i < 8; ++i) d[q] |= encode_sr(value_bits<SRC_BF16>(c[q], i), inv, rnd[8 * q + i]) << (4 * i);
    }
  } else {
#pragma unroll
    for (int q = 0; q < 4; ++q) d[q] = encode8<SRC_BF16>(c[q], sb);
  }
  return make_uint4(d[0], d[1], d[2], d[3]);
}

// Rowwise: one lane per block, as the 8-bit rowwise kernel (64 or 128 bytes read with 16-byte
// loads, one 16-byte code store; the 64 scale bytes of a wave are one run).
template <int SRC_BF16, bool SR, int R>
__global__ __launch_bounds__(kThreads) void k_quant4_rows(const char* __restrict__ src, int64_t ld_src, int64_t K,
                                                         int64_t nb, int64_t nblocks, uint8_t* __restrict__ codes,
                                                         int64_t ld_codes, uint8_t* __restrict__ scales,
                                                         int64_t ld_scales, uint64_t seed) {
  constexpr int ES = SRC_BF16 ? 2 : 4;
  const int64_t stride = (int64_t)gridDim.x * kThreads;
  for (int64_t g = (int64_t)blockIdx.x * kThreads + threadIdx.x; g < nblocks; g += stride) {
    const int64_t row = nblocks <= 0xFFFFFFFF ? (int64_t)((uint32_t)g / (uint32_t)nb) : g / nb;
    const int64_t b = g - row * nb;
    const char* line = src + row * ld_src * ES;
    Chunk<SRC_BF16> c[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) load_chunk<SRC_BF16>(c[q], line, 32 * b + 8 * q, K);
    uint32_t amax = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t a = chunk_abs_max<SRC_BF16>(c[q]);
      amax = amax > a ? amax : a;
    }
    const uint32_t sb = scale_byte<R>(amax);
    *reinterpret_cast<uint4*>(codes + row * ld_codes + 16 * b) = encode32<SRC_BF16, SR>(c, sb, (uint64_t)g, seed);
    scales[row * ld_scales + b] = (uint8_t)sb;
  }
}

// Columnwise, and both orientations from one read (ROWS).  A workgroup takes a tile of 128
// rows x 128 columns: thread t's q-th chunk (8 values) is row t / 16 + 16 q, chunk t % 16, so
// a quad holds one 32-value row block (reduced with DPP) and the tile goes to LDS with the
// dword index of row r XOR SWZ * ((r >> 5) & 3) (the layout of the 8-bit dual kernel: the four
// blocks of a column that a half-wave reads back fall on different banks).  Lane 4c + kb of
// wave w then takes column 64u + 16w + c, block kb.  Tiles are walked in groups of 8 x 32
// tiles and dealt to the XCDs in contiguous chunks.
template <int SRC_BF16, bool ROWS, bool SR, int R>
__global__ __launch_bounds__(kThreads) void k_quant4_tile(const char* __restrict__ src, int64_t rows, int64_t cols,
                                                         int64_t ld_src, uint8_t* __restrict__ rcodes, int64_t ld_rc,
                                                         uint8_t* __restrict__ rscales, int64_t ld_rs,
                                                         uint8_t* __restrict__ ccodes, int64_t ld_cc,
                                                         uint8_t* __restrict__ cscales, int64_t ld_cs, int64_t gx,
                                                         int64_t ntiles, int64_t per_xcd, uint64_t seed) {
  constexpr int ES = SRC_BF16 ? 2 : 4;
  constexpr int RW = 128 * ES / 4;   // dwords per tile row
  constexpr int CW = 8 * ES / 4;     // dwords per chunk
  constexpr int SWZ = 2 * ES;        // dwords of a half-wave's 8 columns
  extern __shared__ __align__(16) uint32_t tile[];
  const int tid = threadIdx.x;
  const int lane = tid & 63, wv = tid >> 6;
  const int wg = workgroup_at(blockIdx.x, blockIdx.y);
  const int64_t t = (wg % kXcds) * per_xcd + wg / kXcds;
  if (wg / kXcds >= per_xcd || t >= ntiles) return;  // the whole workgroup, before any barrier
  const int64_t gy = ntiles / gx;
  const int64_t band = t / (8 * gx), rem = t - band * 8 * gx;
  const int64_t hb = gy - 8 * band < 8 ? gy - 8 * band : 8;
  const int64_t grp = rem / (32 * hb), r2 = rem - grp * 32 * hb;
  const int64_t wdt = gx - 32 * grp < 32 ? gx - 32 * grp : 32;
  const int64_t y = 8 * band + r2 / wdt, x = 32 * grp + r2 % wdt;
  const int64_t c0 = 128 * x, r0 = 128 * y;
  const int64_t nb_r = (cols + 31) / 32, nb_c = (rows + 31) / 32;
  const int chunk = tid & 15;
  const int64_t cc = c0 + 8 * chunk;
  Chunk<SRC_BF16> chs[8];
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int64_t r = r0 + (tid >> 4) + 16 * q;
    load_chunk<SRC_BF16>(chs[q], src + r * ld_src * ES, cc, r < rows ? cols : 0);
  }
#pragma unroll
  for (int q = 0; q < 8; ++q) {
    const int row = (tid >> 4) + 16 * q;
    const Chunk<SRC_BF16>& ch = chs[q];
    const int sw = SWZ * ((row >> 5) & 3);
#pragma unroll
    for (int h = 0; h < ES / 2; ++h)
      *reinterpret_cast<uint4*>(&tile[row * RW + ((CW * chunk + 4 * h) ^ sw)]) =
          make_uint4(ch.w[4 * h], ch.w[4 * h + 1], ch.w[4 * h + 2], ch.w[4 * h + 3]);
    if (ROWS) {
      const uint32_t sb = scale_byte<R>(mxblock::quad_max(chunk_abs_max<SRC_BF16>(ch)));
      const uint32_t d = encode8<SRC_BF16>(ch, sb);
      const int64_t r = r0 + row;
      if (r < rows && cc < 32 * nb_r) {
        *reinterpret_cast<uint32_t*>(rcodes + r * ld_rc + cc / 2) = d;
        if ((chunk & 3) == 0) rscales[r * ld_rs + (cc >> 5)] = (uint8_t)sb;
      }
    }
  }
  __syncthreads();
  const int kb = lane & 3;
  const int64_t b = 4 * y + kb;
  if (b >= nb_c) return;                             // no barrier follows
#pragma unroll 1
  for (int u = 0; u < 2; ++u) {
    const int cl = 64 * u + 16 * wv + (lane >> 2);
    const int64_t col = c0 + cl;
    if (col >= cols) break;
    Chunk<SRC_BF16> c[4];
#pragma unroll
    for (int i = 0; i < 32; ++i) {
      const int row = 32 * kb + i;
      if (SRC_BF16) {
        const uint32_t v = reinterpret_cast<const uint16_t*>(tile)[2 * (row * RW + ((cl >> 1) ^ (SWZ * kb))) + (cl & 1)];
        if (i & 1)
          c[i >> 3].w[(i & 7) >> 1] |= v << 16;
        else
          c[i >> 3].w[(i & 7) >> 1] = v;
      } else {
        c[i >> 3].w[i & 7] = tile[row * RW + (cl ^ (SWZ * kb))];
      }
    }
    uint32_t amax = 0;
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const uint32_t a = chunk_abs_max<SRC_BF16>(c[q]);
      amax = amax > a ? amax : a;
    }
    const uint32_t sb = scale_byte<R>(amax);
    *reinterpret_cast<uint4*>(ccodes + col * ld_cc + 16 * b) =
        encode32<SRC_BF16, SR>(c, sb, (uint64_t)col * (uint64_t)nb_c + (uint64_t)b, seed);
    cscales[col * ld_cs + b] = (uint8_t)sb;
  }
}

template <int SRC_BF16, bool ROWS, bool SR, int R>
hipError_t launch_tile(const void* src, int64_t rows, int64_t cols, int64_t ld_src, uint8_t* rc, int64_t ld_rc,
                       uint8_t* rs, int64_t ld_rs, uint8_t* cc, int64_t ld_cc, uint8_t* cs, int64_t ld_cs,
                       uint64_t seed, hipStream_t st) {
  const int64_t gx = (cols + 127) / 128, gy = (rows + 127) / 128, n = gx * gy;
  const int64_t per_xcd = (n + kXcds - 1) / kXcds;
  if (kXcds * per_xcd > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int lds = 128 * 128 * (SRC_BF16 ? 2 : 4);
  const Grid grid = grid_of(kXcds * per_xcd);
  hipLaunchKernelGGL((k_quant4_tile<SRC_BF16, ROWS, SR, R>), dim3(grid.x, grid.y), dim3(kThreads), lds, st,
                     (const char*)src, rows, cols, ld_src, rc, ld_rc, rs, ld_rs, cc, ld_cc, cs, ld_cs, gx, n, per_xcd,
                     seed);
  return hipGetLastError();
}

template <int SRC_BF16, bool SR, int R>
hipError_t launch_rows(const void* src, int64_t rows, int64_t K, int64_t ld_src, uint8_t* codes, int64_t ld_codes,
                       uint8_t* scales, int64_t ld_scales, uint64_t seed, hipStream_t st) {
  const int64_t nb = (K + 31) / 32, n = rows * nb;
  const int64_t want = (n + kThreads - 1) / kThreads, cap = (int64_t)device_cu_count() * 256;
  hipLaunchKernelGGL((k_quant4_rows<SRC_BF16, SR, R>), dim3((unsigned)(want < cap ? want : cap)), dim3(kThreads), 0, st,
                     (const char*)src, ld_src, K, nb, n, codes, ld_codes, scales, ld_scales, seed);
  return hipGetLastError();
}

template <int SRC_BF16, bool SR, int R>
hipError_t launch_axis(const void* src, int64_t rows, int64_t cols, int64_t ld_src, bool colwise, uint8_t* codes,
                       int64_t ld_codes, uint8_t* scales, int64_t ld_scales, uint64_t seed, hipStream_t st) {
  if (colwise)
    return launch_tile<SRC_BF16, false, SR, R>(src, rows, cols, ld_src, nullptr, 0, nullptr, 0, codes, ld_codes, scales,
                                               ld_scales, seed, st);
  return launch_rows<SRC_BF16, SR, R>(src, rows, cols, ld_src, codes, ld_codes, scales, ld_scales, seed, st);
}

// Dequantize: chunks of E = 16 / sizeof(output) elements, one 16-byte store each; lane t of a
// wave takes chunks t, t + 64, ... of the wave's 256, so every access of the wave is one
// contiguous run and all its loads are in flight before its first store.  A chunk at the end
// of a line whose length is no multiple of E is stored element by element.
template <int OUT_BF16>
__global__ __launch_bounds__(kThreads) void k_dequant4(const uint8_t* __restrict__ codes, int64_t ld_codes,
                                                      const uint8_t* __restrict__ scales, int64_t ld_scales, int64_t K,
                                                      int64_t cpl, int64_t nchunks, char* __restrict__ dst,
                                                      int64_t ld_dst) {
  constexpr int E = OUT_BF16 ? 8 : 4;
  constexpr int ES = OUT_BF16 ? 2 : 4;
  constexpr int NC = 4;
  const int lane = threadIdx.x & 63;
  const int64_t first = ((int64_t)blockIdx.x * (kThreads / 64) + (threadIdx.x >> 6)) * (64 * NC) + lane;
  uint32_t w[NC], sb[NC];
  int64_t l[NC], k[NC];
#pragma unroll
  for (int q = 0; q < NC; ++q) {
    const int64_t c = first + 64 * q;
    w[q] = sb[q] = 0;
    l[q] = nchunks <= 0xFFFFFFFF ? (int64_t)((uint32_t)c / (uint32_t)cpl) : c / cpl;
    k[q] = E * (c - l[q] * cpl);
    if (c < nchunks) {
      // a line holds 16 * ceil(K / 32) >= (k + E + 1) / 2 bytes, so the chunk's bytes are there
      const uint8_t* p = codes + l[q] * ld_codes + k[q] / 2;
      w[q] = OUT_BF16 ? *reinterpret_cast<const uint32_t*>(p) : (uint32_t)*reinterpret_cast<const uint16_t*>(p);
      sb[q] = scales[l[q] * ld_scales + (k[q] >> 5)];
    }
  }
#pragma unroll
  for (int q = 0; q < NC; ++q) {
    if (first + 64 * q >= nchunks) break;
    const float s = e8m0_to_f32(sb[q]);
    uint32_t o[4];
    if (OUT_BF16) {
      decode8_bf16(w[q], s, o);
    } else {
      float f[4];
      decode4_f32(w[q], s, f);
#pragma unroll
      for (int i = 0; i < 4; ++i) o[i] = __float_as_uint(f[i]);
    }
    char* p = dst + (l[q] * ld_dst + k[q]) * ES;
    if (k[q] + E <= K) {
      __builtin_memcpy(p, o, 16);
    } else {
#pragma unroll
      for (int i = 0; i < E; ++i)
        if (k[q] + i < K) {
          if (OUT_BF16)
            reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(o[i >> 1] >> (16 * (i & 1)));
          else
            reinterpret_cast<uint32_t*>(p)[i] = o[i & 3];
        }
    }
  }
}

}  // namespace

hipError_t launch_quant4(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, bool colwise,
                         int rule, bool sr, uint64_t seed, uint8_t* codes, int64_t ld_codes, uint8_t* scales,
                         int64_t ld_scales, hipStream_t st) {
#define MXQ_Q4(B, S, R) \
  return launch_axis<B, S, R>(src, rows, cols, ld_src, colwise, codes, ld_codes, scales, ld_scales, seed, st)
  if (sr) {
    if (src_bf16) MXQ_Q4(1, true, kRuleCeil);
    MXQ_Q4(0, true, kRuleCeil);
  }
  if (rule == kRuleOcp) {
    if (src_bf16) MXQ_Q4(1, false, kRuleOcp);
    MXQ_Q4(0, false, kRuleOcp);
  }
  if (src_bf16) MXQ_Q4(1, false, kRuleCeil);
  MXQ_Q4(0, false, kRuleCeil);
#undef MXQ_Q4
}

hipError_t launch_quant4_dual(const void* src, int src_bf16, int64_t rows, int64_t cols, int64_t ld_src, uint8_t* rc,
                              int64_t ld_rc, uint8_t* rs, int64_t ld_rs, uint8_t* cc, int64_t ld_cc, uint8_t* cs,
                              int64_t ld_cs, hipStream_t st) {
  if (src_bf16)
    return launch_tile<1, true, false, kRuleCeil>(src, rows, cols, ld_src, rc, ld_rc, rs, ld_rs, cc, ld_cc, cs, ld_cs,
                                                  0, st);
  return launch_tile<0, true, false, kRuleCeil>(src, rows, cols, ld_src, rc, ld_rc, rs, ld_rs, cc, ld_cc, cs, ld_cs, 0,
                                                st);
}

hipError_t launch_dequant4(const uint8_t* codes, int64_t ld_codes, const uint8_t* scales, int64_t ld_scales, int64_t L,
                           int64_t K, void* dst, int dst_bf16, int64_t ld_dst, hipStream_t st) {
  const int64_t e = dst_bf16 ? 8 : 4, cpl = (K + e - 1) / e, n = L * cpl;
  const int64_t blocks = (n + 1023) / 1024;
  if (blocks > 0x7FFFFFFF) return hipErrorInvalidValue;
  if (dst_bf16)
    hipLaunchKernelGGL((k_dequant4<1>), dim3((unsigned)blocks), dim3(kThreads), 0, st, codes, ld_codes, scales,
                       ld_scales, K, cpl, n, (char*)dst, ld_dst);
  else
    hipLaunchKernelGGL((k_dequant4<0>), dim3((unsigned)blocks), dim3(kThreads), 0, st, codes, ld_codes, scales,
                       ld_scales, K, cpl, n, (char*)dst, ld_dst);
  return hipGetLastError();
}

}  // namespace mxq
