// gemm_fp4_tile.hip -- the product of two MXFP4 matrices in 256 x 256 tiles on the scaled FP4
// matrix cores of gfx950.
//
// v_mfma_scale_f32_32x32x64_f8f6f4 with both operands E2M1: lane l = 32 g + i supplies the 16
// bytes of MX block g of row i (A) or column i (B) of the 64-wide step and, through opsel, its
// E8M0 byte; the sums of a block are exact (multiples of 1/4), blocks combine in FP32.  One
// issues every 33 cycles per SIMD; 1024 SIMDs of them on random codes run at 6.0-6.4 PFLOP/s
// (the clock drops under the switching load), the ceiling of this kernel.
//
// The schedule is the ping-pong of the 8-bit kernel (gemm_fp8.hip) at twice the K per byte:
// eight waves, waves w and w + 4 on one SIMD, group 0 (waves 0-3) owning rows 0-127 of the
// tile and group 1 rows 128-255, a wave 128 x 64 (4 x 2 accumulators of 32 x 32).  A K step is
// 64 bytes = 128 codes = 4 blocks of every row: both tiles' 32 KiB go to one of four LDS stages
// by LDS DMA, three steps ahead, a row's 16-byte block c at c ^ ((row >> 2) & 3), so fragment
// reads are conflict free.  The two groups alternate between reading a step's fragments and
// scales from LDS and issuing its 16 MFMAs, with the DMA of a later step between them.  Scale
// rows travel 16 bytes (4 steps) at a time into a two-slot ring.  Reads past a row's codes or
// the matrix's rows return zero through the descriptors; in the last, partial step codes at
// k >= K are zeroed and the scale of a block >= nb is 127.
//
// What bounds it: power and the movement of operands.  8192 x 4096 x 4096 takes 75-81 us (3.4-3.7 PFLOP/s),
// 16384 deep 318 us at a clock that falls to 1.7 GHz; there the MFMAs are busy 55 % of the cycles.  MFMAs alone, on
// operands that stay in registers, hold 6.4-6.6 PFLOP/s for 30 ms (random codes; zeros 9.7).  Of
// the 318 us a copy of this kernel without the DMA needs 262, without the LDS reads of fragments
// 324, without both 250, with all codes zero 221: taking a step's scales four at a time (their 4-byte
// reads are the only LDS reads with bank conflicts), DMA in lines of 128 bytes and DMA beside the LDS
// reads instead of between the MFMAs gain nothing.
#include "fp4_ranges.hpp"
#include "gemm_common.hpp"

namespace mxq {
namespace {
namespace fp4t {

constexpr int BM = 256, BN = 256;
constexpr int kThreads = 512;
constexpr int kStages = 4;
constexpr int kCodeBytes = 256 * 64;            // one operand's codes in one stage
constexpr int kOffB = kCodeBytes;
constexpr int kStageBytes = 2 * kCodeBytes;     // 32 KiB
constexpr int kOffScale = kStages * kStageBytes;
constexpr int kScaleSlot = 2 * 256 * 16;        // A then B: 256 rows x 16 bytes each
constexpr int kOffJunk = kOffScale + 2 * kScaleSlot;    // target of the idle scale loads
constexpr int kLdsBytes = kOffJunk + 1024;               // 145 KiB
constexpr int kEpiWaveBytes = 16384;            // per-wave epilogue staging (in the code stages)

struct Dma {
  uint64_t a_base, b_base, s_base;   // tile row 0 of X codes, W codes, this wave's scales
  uint32_t a_bytes, b_bytes, s_bytes;
  uint32_t voff_a0, voff_a1, voff_b0, voff_b1, voff_s;
  uint32_t lds_a, lds_b, lds_s;      // LDS destinations (code stage 0, scale slot 0)
  uint32_t lds_junk;
  int T;
};

// Every step's DMA is 5 loads per wave: two 16-row pieces of each code tile and the scales, which
// every fourth step are this wave's 64 scale rows of the next four steps and else an empty load
// into a junk area, so the waits below are constants.  Steps >= T get an empty range.
constexpr int kLoadsPerStep = 5;
struct StepDma {
  v4i ra, rb;
  uint32_t so;
};

__device__ __forceinline__ StepDma step_dma(const Dma& d, int s) {
  const bool live = s < d.T;
  const uint32_t kb = live ? 64u * (uint32_t)s : 0u;
  return StepDma{rsrc_of(d.a_base + kb, live ? d.a_bytes - kb : 0u), rsrc_of(d.b_base + kb, live ? d.b_bytes - kb : 0u),
                 (uint32_t)(s & 3) * kStageBytes};
}

__device__ __forceinline__ void issue_scales(const Dma& d, int s) {
  const bool real = (s & 3) == 0;
  const bool live = real && s < d.T;
  const uint32_t ub = live ? 4u * (uint32_t)s : 0u;    // 16 bytes per 4 steps
  const v4i rs = rsrc_of(d.s_base + ub, live ? d.s_bytes - ub : 0u);
  dma16(real ? d.lds_s + (uint32_t)((s >> 2) & 1) * kScaleSlot : d.lds_junk, d.voff_s, rs);
}

__device__ __forceinline__ void issue_step(const Dma& d, int s) {
  const StepDma sd = step_dma(d, s);
  dma16(d.lds_a + sd.so, d.voff_a0, sd.ra);
  dma16(d.lds_a + sd.so + 1024, d.voff_a1, sd.ra);
  dma16(d.lds_b + sd.so, d.voff_b0, sd.rb);
  dma16(d.lds_b + sd.so + 1024, d.voff_b1, sd.rb);
  issue_scales(d, s);
}

#pragma clang diagnostic push
#pragma clang diagnostic ignored "-Winline-asm"
// dma16 placed between two MFMAs: it names `after` (an operand of the MFMAs before it) and
// `before` (an operand of the MFMAs after it) as read-write operands it never touches.
template <typename V>
__device__ __forceinline__ void dma16_between(uint32_t lds, uint32_t voff, v4i rsrc, V& after, V& before) {
  asm volatile("s_mov_b32 m0, %2\n\tbuffer_load_dwordx4 %3, %4, 0 offen lds"
               : "+v"(after), "+v"(before)
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
template <typename V>
__device__ __forceinline__ void dma16_after(uint32_t lds, uint32_t voff, v4i rsrc, V& after) {
  asm volatile("s_mov_b32 m0, %1\n\tbuffer_load_dwordx4 %2, %3, 0 offen lds"
               : "+v"(after)
               : "s"(__builtin_amdgcn_readfirstlane(lds)), "v"(voff), "s"(rsrc)
               : "memory", "m0");
}
#pragma clang diagnostic pop

__device__ __forceinline__ v8i widen(v4i v) { return v8i{v[0], v[1], v[2], v[3], 0, 0, 0, 0}; }

template <bool TAIL>
__global__ __launch_bounds__(kThreads, 1) void k_gemm4_tile(int M, int N, int K, int tiles_m, int tiles_n,
                                                           const uint8_t* __restrict__ xc, int64_t ld_x,
                                                           const uint8_t* __restrict__ xs, int64_t ld_xs,
                                                           const uint8_t* __restrict__ wc, int64_t ld_w,
                                                           const uint8_t* __restrict__ ws, int64_t ld_ws,
                                                           const GemmEpilogue ep) {
  const int wg = workgroup_at(blockIdx.x, blockIdx.y);
  if (blockIdx.y > 0 && wg >= tiles_m * tiles_n) return;
  int tm, tn;
  tile_of(wg, tiles_m, tiles_n, tm, tn);
  const int m0 = tm * BM, n0 = tn * BN;

  const int lane = threadIdx.x & 63;
  const int wid = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int gp = wid >> 2, wq = wid & 3;
  const int li = lane & 31, lg = lane >> 5;
  const int nb = (K + 31) / 32;
  const int T = (K + 127) / 128;
  const int rows_a = min(BM, M - m0), rows_b = min(BN, N - n0);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(lds_ptr_t)smem;

  // ---- DMA set-up: wave w loads rows 32w..32w+31 of both code tiles; load n covers rows
  //      32w + 16n + lane/4, physical block lane & 3 holding logical block
  //      (lane & 3) ^ ((row >> 2) & 3).  Scales: waves 0-3 rows 64w + lane of X, waves 4-7
  //      rows 64(w-4) + lane of W.
  Dma d;
  {
    d.T = T;
    d.a_base = (uint64_t)(uintptr_t)(xc + (int64_t)m0 * ld_x);
    d.b_base = (uint64_t)(uintptr_t)(wc + (int64_t)n0 * ld_w);
    d.a_bytes = (uint32_t)((int64_t)(rows_a - 1) * ld_x + 16 * nb);
    d.b_bytes = (uint32_t)((int64_t)(rows_b - 1) * ld_w + 16 * nb);
    const int drow = 32 * wid + (lane >> 2);
    const int dblock = (lane & 3) ^ ((lane >> 4) & 3);
    d.voff_a0 = (uint32_t)(drow * ld_x + 16 * dblock);
    d.voff_a1 = d.voff_a0 + (uint32_t)(16 * ld_x);
    d.voff_b0 = (uint32_t)(drow * ld_w + 16 * dblock);
    d.voff_b1 = d.voff_b0 + (uint32_t)(16 * ld_w);
    d.lds_a = lds0 + (uint32_t)(32 * wid) * 64;
    d.lds_b = lds0 + kOffB + (uint32_t)(32 * wid) * 64;
    d.lds_junk = lds0 + kOffJunk;
    // scale rows are read in 4-byte words, none past the word that holds the last byte
    const int nb4 = (nb + 3) & ~3;
    const int srow = 64 * (wid & 3) + lane;
    if (wid < 4) {
      d.s_base = (uint64_t)(uintptr_t)(xs + (int64_t)m0 * ld_xs);
      d.s_bytes = (uint32_t)((int64_t)(rows_a - 1) * ld_xs + nb4);
      d.voff_s = (uint32_t)(srow * ld_xs);
      d.lds_s = lds0 + kOffScale + (uint32_t)(64 * wid) * 16;
    } else {
      d.s_base = (uint64_t)(uintptr_t)(ws + (int64_t)n0 * ld_ws);
      d.s_bytes = (uint32_t)((int64_t)(rows_b - 1) * ld_ws + nb4);
      d.voff_s = (uint32_t)(srow * ld_ws);
      d.lds_s = lds0 + kOffScale + 4096 + (uint32_t)(64 * (wid - 4)) * 16;
    }
  }

  // ---- fragment read addresses (stage 0) of the step's halves h: block 2h + g of the row;
  //      tile f / fj adds 2048 bytes.  Scale read addresses (slot 0): row * 16, tile f / fj
  //      adds 512 bytes.
  const uint32_t xsw = (uint32_t)((li >> 2) & 3);
  uint32_t ra[2], rb[2];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    const uint32_t c = (uint32_t)(2 * h + lg);
    ra[h] = (uint32_t)(gp * 128 + li) * 64 + ((c ^ xsw) << 4);
    rb[h] = kOffB + (uint32_t)(wq * 64 + li) * 64 + ((c ^ xsw) << 4);
  }
  const uint32_t rsa = kOffScale + (uint32_t)(gp * 128 + li) * 16;
  const uint32_t rsb = kOffScale + 4096 + (uint32_t)(wq * 64 + li) * 16;

  v16f acc[4][2];
#pragma unroll
  for (int i = 0; i < 4; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;

  v4i fa[2][4], fb[2][2];
  uint32_t sa[4], sb[2];

  // memory phase of step s: its fragments and scales, then wait for this wave's DMA of step
  // s + 1; only the DMA of step s + 2 stays in flight
  auto memory_phase = [&](int s, auto last) {
    const uint32_t so = (uint32_t)(s & 3) * kStageBytes;
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int f = 0; f < 4; ++f) fa[h][f] = lds16(ra[h] + so, 2048 * f);
#pragma unroll
      for (int f = 0; f < 2; ++f) fb[h][f] = lds16(rb[h] + so, 2048 * f);
    }
    // the step's four scale bytes of a fragment row; lane group g uses byte g of each half
    const uint32_t ss = (uint32_t)((s >> 2) & 1) * kScaleSlot + 4u * (uint32_t)(s & 3);
#pragma unroll
    for (int f = 0; f < 4; ++f) sa[f] = *reinterpret_cast<const uint32_t*>(smem + rsa + ss + 512 * f);
#pragma unroll
    for (int f = 0; f < 2; ++f) sb[f] = *reinterpret_cast<const uint32_t*>(smem + rsb + ss + 512 * f);
    if (decltype(last)::value) {
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int left = K - (128 * s + 64 * h + 32 * lg);    // codes of this lane's block
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int keep = left - 8 * e;
          const uint32_t m = keep >= 8 ? 0xFFFFFFFFu : (keep <= 0 ? 0u : ((1u << (4 * keep)) - 1u));
#pragma unroll
          for (int f = 0; f < 4; ++f) fa[h][f][e] = (int)((uint32_t)fa[h][f][e] & m);
#pragma unroll
          for (int f = 0; f < 2; ++f) fb[h][f][e] = (int)((uint32_t)fb[h][f][e] & m);
        }
      }
#pragma unroll
      for (int b = 0; b < 4; ++b)
        if (4 * s + b >= nb) {
          const uint32_t keep = ~(0xFFu << (8 * b)), one = 127u << (8 * b);
#pragma unroll
          for (int f = 0; f < 4; ++f) sa[f] = (sa[f] & keep) | one;
#pragma unroll
          for (int f = 0; f < 2; ++f) sb[f] = (sb[f] & keep) | one;
        }
    }
#pragma unroll
    for (int f = 0; f < 4; ++f) sa[f] >>= 8 * lg;
#pragma unroll
    for (int f = 0; f < 2; ++f) sb[f] >>= 8 * lg;
    if (decltype(last)::value)
      wait_vm<0>();    // also the empty loads of steps T and T+1
    else
      wait_vm<kLoadsPerStep>();
  };

  // Compute phase of step s: 16 MFMAs, with this wave's DMA of step s + 3 (whose stage was last
  // read in the phase before) between them; the last step issues none.  The empty volatile
  // asm statements make the MFMAs take their operands only after the barrier that opens the
  // phase.
  auto compute_phase = [&](int s, auto with_dma) {
    constexpr bool DMA = decltype(with_dma)::value;
    StepDma sd;
    if (DMA) {
      sd = step_dma(d, s + 3);
      issue_scales(d, s + 3);
    }
#pragma unroll
    for (int h = 0; h < 2; ++h)
      asm volatile("" : "+v"(fa[h][0]), "+v"(fa[h][1]), "+v"(fa[h][2]), "+v"(fa[h][3]), "+v"(fb[h][0]), "+v"(fb[h][1]));
    asm volatile("" : "+v"(sa[0]), "+v"(sa[1]), "+v"(sa[2]), "+v"(sa[3]), "+v"(sb[0]), "+v"(sb[1]));
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int fi = 0; fi < 4; ++fi) {
#pragma unroll
        for (int fj = 0; fj < 2; ++fj)
          acc[fi][fj] = h == 0 ? __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                     widen(fb[h][fj]), widen(fa[h][fi]), acc[fi][fj], 4, 4, 0, (int)sb[fj], 0, (int)sa[fi])
                               : __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
                                     widen(fb[h][fj]), widen(fa[h][fi]), acc[fi][fj], 4, 4, 2, (int)sb[fj], 2, (int)sa[fi]);
        if (DMA && (fi & 1)) {
          // one of the step's four code loads after every fourth MFMA
          const int n = 2 * h + (fi >> 1);
          const uint32_t lds = (n < 2 ? d.lds_a : d.lds_b) + sd.so + 1024 * (n & 1);
          const uint32_t voff = n == 0 ? d.voff_a0 : n == 1 ? d.voff_a1 : n == 2 ? d.voff_b0 : d.voff_b1;
          if (n == 3)
            dma16_after(lds, voff, sd.rb, fa[1][3]);
          else
            dma16_between(lds, voff, n < 2 ? sd.ra : sd.rb, fa[h][fi], n == 1 ? fa[1][0] : fa[h][fi + 1 < 4 ? fi + 1 : 3]);
        }
      }
  };

  // ---- prologue: steps 0..2 in flight, step 0 landed everywhere
#pragma unroll
  for (int s = 0; s < 3; ++s) issue_step(d, s);
  wait_vm<2 * kLoadsPerStep>();
  lds_barrier();
  if (gp == 1) lds_barrier();   // group 1 runs one phase behind group 0

  auto step = [&](int s, auto last) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    memory_phase(s, last);
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
    __builtin_amdgcn_sched_barrier(0);
    compute_phase(s, std::integral_constant<bool, !decltype(last)::value>());
    __builtin_amdgcn_sched_barrier(0);
    lds_barrier();
  };
  if constexpr (TAIL) {
    for (int s = 0; s < T - 1; ++s) step(s, std::false_type());
    step(T - 1, std::true_type());
  } else {
    for (int s = 0; s < T; ++s) step(s, std::false_type());
    wait_vm<0>();
    lds_barrier();
  }
  if (gp == 0) lds_barrier();   // matches group 1's extra barrier: all LDS reads are done

  // ---- epilogue: v = act(alpha * acc + bias[col]) in place; y = v rounded once to its type.
  //      Lane (g, i) holds Y[row 32 fi + i][col 32 fj + 8 q + 4 g + e] in acc[fi][fj][4 q + e]
  //      (rows and columns relative to the wave's 128x64 block).
  const int wrow0 = m0 + gp * 128, wcol0 = n0 + wq * 64;
  {
    const bool has_bias = ep.bias != nullptr;
    const __amdgpu_buffer_rsrc_t brs = bias_rsrc(ep.bias, N);
    typedef float v4f __attribute__((ext_vector_type(4)));
#pragma unroll
    for (int fj = 0; fj < 2; ++fj)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const v4f b = __builtin_bit_cast(
            v4f, __builtin_amdgcn_raw_buffer_load_b128(brs, 4 * (wcol0 + 32 * fj + 8 * q + 4 * lg), 0, 0));
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const int col = wcol0 + 32 * fj + 8 * q + 4 * lg + e;
          const float bv = (has_bias && col < N) ? b[e] : -0.0f;
#pragma unroll
          for (int fi = 0; fi < 4; ++fi)
            acc[fi][fj][4 * q + e] = __builtin_fmaf(ep.alpha, acc[fi][fj][4 * q + e], bv);
        }
      }
    if (ep.act) {
#pragma unroll
      for (int fi = 0; fi < 4; ++fi)
#pragma unroll
        for (int fj = 0; fj < 2; ++fj)
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[fi][fj][r] = silu(acc[fi][fj][r]);
    }
  }
  // stage the block in this wave's LDS region as row-major rows of 64 values with the 16-byte
  // chunk index XOR (row & 7), then store whole 16-byte row pieces (E = bytes per value); where the tile
  // or the matrix ends, or y is not aligned, piece by piece with its bounds (element by element, as the
  // fragments lie, a ragged tile took 15 us longer than a whole one)
  const bool whole = ep.y_vec16 && M - m0 >= BM && N - n0 >= BN;
  auto store_staged = [&](auto e_c) {
    constexpr int E = decltype(e_c)::value;
    constexpr int RB = 64 * E;                       // bytes per staged row
    constexpr int CPR = RB / 16;                     // 16-byte chunks per row
    constexpr int RP = kEpiWaveBytes / RB;           // rows per pass: 128 (bf16) or 64 (fp32)
    constexpr int FPP = RP / 32;                     // fragment rows per pass
    const uint32_t wbase = (uint32_t)wid * kEpiWaveBytes;
#pragma unroll
    for (int pass = 0; pass < 128 / RP; ++pass) {
#pragma unroll
      for (int fj = 0; fj < 2; ++fj)
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          const int c0 = 32 * fj + 8 * q + 4 * lg;   // first of this lane's 4 columns
#pragma unroll
          for (int fl = 0; fl < FPP; ++fl) {
            const int fi = pass * FPP + fl;
            const int row = 32 * fl + li;
            const uint32_t byte = (uint32_t)(c0 * E);
            const uint32_t chunk = (byte >> 4) ^ (uint32_t)(row & (CPR - 1) & 7);
            const uint32_t addr = wbase + (uint32_t)row * RB + (chunk << 4) + (byte & 15);
            if (E == 2) {
              typedef uint32_t v2u __attribute__((ext_vector_type(2)));
              v2u p;
              p[0] = pack_bf16(acc[fi][fj][4 * q + 0], acc[fi][fj][4 * q + 1]);
              p[1] = pack_bf16(acc[fi][fj][4 * q + 2], acc[fi][fj][4 * q + 3]);
              *reinterpret_cast<v2u*>(smem + addr) = p;
            } else {
              typedef float v4f __attribute__((ext_vector_type(4)));
              v4f p;
#pragma unroll
              for (int e = 0; e < 4; ++e) p[e] = acc[fi][fj][4 * q + e];
              *reinterpret_cast<v4f*>(smem + addr) = p;
            }
          }
        }
      // read back 16 bytes per lane: 64 lanes cover 1024 bytes = 1024 / RB rows
      constexpr int RPI = 1024 / RB;
#pragma unroll
      for (int it = 0; it < RP / RPI; ++it) {
        const int row = it * RPI + lane / CPR;
        const int c = lane % CPR;
        const uint32_t addr = wbase + (uint32_t)row * RB + (uint32_t)((c ^ (row & (CPR - 1) & 7)) << 4);
        const v4i v = *reinterpret_cast<const v4i*>(smem + addr);
        const int gr = wrow0 + pass * RP + row, gc = wcol0 + (16 / E) * c;
        uint8_t* dst = reinterpret_cast<uint8_t*>(ep.y) + ((int64_t)gr * ep.ld_y + gc) * E;
        if (whole) {
          *reinterpret_cast<v4i*>(dst) = v;
        } else if (gr < M) {
          if (gc + 16 / E <= N) {
            __builtin_memcpy(dst, &v, 16);
          } else {
#pragma unroll
            for (int e = 0; e < 16 / E; ++e)
              if (gc + e < N) {
                if (E == 2)
                  reinterpret_cast<uint16_t*>(dst)[e] = (uint16_t)((uint32_t)v[(e * E) >> 2] >> (16 * (e & 1)));
                else
                  reinterpret_cast<int*>(dst)[e] = v[e & 3];
              }
          }
        }
      }
    }
  };
  if (ep.y_bf16)
    store_staged(std::integral_constant<int, 2>());
  else
    store_staged(std::integral_constant<int, 4>());
}

template <bool TAIL>
hipError_t launch(int64_t M, int64_t N, int64_t K, const uint8_t* xc, int64_t ld_x, const uint8_t* xs, int64_t ld_xs,
                  const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws, const GemmEpilogue& ep,
                  hipStream_t stream) {
  static bool attr_set[64] = {false};
  auto kern = k_gemm4_tile<TAIL>;
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) dev = 0;
  if (!attr_set[dev]) {
    const hipError_t e = hipFuncSetAttribute((const void*)kern, hipFuncAttributeMaxDynamicSharedMemorySize, kLdsBytes);
    if (e != hipSuccess) return e;
    attr_set[dev] = true;
  }
  const int tiles_m = (int)((M + BM - 1) / BM), tiles_n = (int)((N + BN - 1) / BN);
  if ((int64_t)tiles_m * tiles_n > 0x7FFFFFFF) return hipErrorInvalidValue;
  const Grid grid = grid_of((int64_t)tiles_m * tiles_n);
  hipLaunchKernelGGL(kern, dim3(grid.x, grid.y), dim3(kThreads), kLdsBytes, stream, (int)M, (int)N, (int)K, tiles_m, tiles_n,
                     xc, ld_x, xs, ld_xs, wc, ld_w, ws, ld_ws, ep);
  return hipGetLastError();
}

}  // namespace fp4t
}  // namespace

hipError_t launch_gemm_fp4_tile(int64_t M, int64_t N, int64_t K, const uint8_t* xc, int64_t ld_x, const uint8_t* xs,
                                int64_t ld_xs, const uint8_t* wc, int64_t ld_w, const uint8_t* ws, int64_t ld_ws,
                                const GemmEpilogue& ep, hipStream_t stream) {
  if (K % 128 != 0) return fp4t::launch<true>(M, N, K, xc, ld_x, xs, ld_xs, wc, ld_w, ws, ld_ws, ep, stream);
  return fp4t::launch<false>(M, N, K, xc, ld_x, xs, ld_xs, wc, ld_w, ws, ld_ws, ep, stream);
}

}  // namespace mxq
