// moe_fp4_few.hip -- the expert layer where next to no expert has two tokens: two launches, each
// (token, rank) a stream of matrix-vector products of its own.
//
// A wave takes 8 rows of weights at a time: lane l holds block 64 s + l of all of them, so a load
// is 1 KiB of one row and its scales 64 bytes of another, in memory order, straight into registers.
// The values of the lane's block of x are in registers in fp32; 32 codes are 16 conversions with the
// scale (exact) and 32 fp32 fused multiply-adds, 1.5 instructions an element, about 10 TB/s of weights
// on 256 CUs: HBM bounds it.  The 64 lanes' sums are added in a fixed order, halving the rows that a
// lane keeps three times.
//
//   up    a workgroup of 4 waves, a wave 4 columns of I: rows 0 .. 3 gate, 4 .. 7 up.  x goes through LDS
//         once per workgroup.  h is stored in fp32, in the order in which lanes read it going down.
//   down  8 columns of H of a token; the waves share its (rank, 2048 elements of I), each times its
//         expert's share, and their sums are added in LDS in wave order: y is complete.
//
// 35.6 MB of gate and up weights take 12.3 us so (1 token, 4 of 64 experts of 4096 x 2048), 17.8 MB going
// down 8.6; about 5 us of each are the launch, the first loads, which wait for one another, and the sums.
//
// Every wave finds the token's experts itself from the logits, one maximum after the other, while x is on
// its way: that costs it less than waiting for what a launch before would have stored.
#include <math.h>

#include "moe_fp4.hpp"

namespace mxq {
namespace {
namespace few {

constexpr int kSeg = 2048;                   // elements of K that a wave takes at once
constexpr int kRows = 8;                     // rows of weights of a wave
constexpr int kKeys = 4;                     // logits of a lane: E <= 256
constexpr int kUpWaves = 4;
constexpr int kDownWaves = 8;

// The lane's block of 8 rows: codes and scale bytes.
struct Block {
  v4i w[kRows];
  uint32_t s[kRows];

  // N rows into w[q0] .. from `row` (uniform) on; those past `last` repeat it, as lanes past the
  // last block do.
  template <int N>
  __device__ __forceinline__ void ask(int q0, const uint8_t* c, int64_t ld_c, const uint8_t* sc, int64_t ld_s, int row, int last,
                                      int b, int nb) {
    const uint32_t at = (uint32_t)min(b, nb - 1);
    c += row * ld_c;
    sc += row * ld_s;
#pragma unroll
    for (int q = 0; q < N; ++q) {
      w[q0 + q] = *reinterpret_cast<const v4i*>(c + 16u * at);
      s[q0 + q] = sc[at];
      c += row + q < last ? ld_c : 0;
      sc += row + q < last ? ld_s : 0;
    }
  }

  // acc[q] += the dot product of row q's block with x (zero past the last element).
  __device__ __forceinline__ void dot(const float x[32], bool live, float acc[kRows]) const {
#pragma unroll
    for (int q = 0; q < kRows; ++q) {
      const float sc = e8m0_to_f32(live ? s[q] : 127u);
      float even = 0.0f, odd = 0.0f;
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        const uint32_t c = (uint32_t)w[q][d];
        const auto v0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 0);
        const auto v1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 1);
        const auto v2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 2);
        const auto v3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, sc, 3);
        even = __builtin_fmaf(v0[0], x[8 * d], even);
        odd = __builtin_fmaf(v0[1], x[8 * d + 1], odd);
        even = __builtin_fmaf(v1[0], x[8 * d + 2], even);
        odd = __builtin_fmaf(v1[1], x[8 * d + 3], odd);
        even = __builtin_fmaf(v2[0], x[8 * d + 4], even);
        odd = __builtin_fmaf(v2[1], x[8 * d + 5], odd);
        even = __builtin_fmaf(v3[0], x[8 * d + 6], even);
        odd = __builtin_fmaf(v3[1], x[8 * d + 7], odd);
      }
      acc[q] += even + odd;
    }
  }
};

// The sum over the lanes of value lane / 8.
__device__ __forceinline__ float sum_rows(const float v[kRows], int lane) {
  float a[4], b[2];
#pragma unroll
  for (int q = 0; q < 4; ++q) {
    const bool up = lane & 32;
    a[q] = (up ? v[q + 4] : v[q]) + __shfl_xor(up ? v[q] : v[q + 4], 32);
  }
#pragma unroll
  for (int q = 0; q < 2; ++q) {
    const bool up = lane & 16;
    b[q] = (up ? a[q + 2] : a[q]) + __shfl_xor(up ? a[q] : a[q + 2], 16);
  }
  const bool up = lane & 8;
  float c = (up ? b[1] : b[0]) + __shfl_xor(up ? b[0] : b[1], 8);
  c += __shfl_xor(c, 4);
  c += __shfl_xor(c, 2);
  return c + __shfl_xor(c, 1);
}

// Bytes of a slot's hidden values: pieces of 4 in fp32, piece p of block 64 s + l at (8 s + p) * 64 + l.
__host__ __device__ __forceinline__ int64_t hidden_bytes(int64_t I) { return (I + kSeg - 1) / kSeg * kSeg * 4; }

// Byte of x's 16-byte piece q of block b in LDS: the 64 blocks of a read fall on different banks.
__device__ __forceinline__ uint32_t x_at(int b, int q) { return 64u * b + 16u * (q ^ ((b >> 2) & 3)); }

__global__ __launch_bounds__(64 * kUpWaves, 2) void k_moe_few_up(const MoeArgs a) {
  const int slot = blockIdx.x / a.tiles, tile = blockIdx.x % a.tiles;
  const int t = slot / a.k, rank = slot % a.k;
  const int lane = threadIdx.x & 63;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nb = (a.H + 31) / 32, segs = (a.H + kSeg - 1) / kSeg;
  Logits<kKeys> lg;
  lg.load(a, t, lane);
  // x: thread's 16-byte pieces threadIdx.x + 256 n, the first two on their way while experts are chosen
  const uint8_t* xr = a.x + t * a.ld_x;
  auto x_piece = [&](int n) {
    const int k = 8 * ((int)threadIdx.x + 256 * n);
    v4i v = {0, 0, 0, 0};
    if (k + 8 <= a.H) {
      __builtin_memcpy(&v, xr + 2 * k, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 8; ++e)
        if (k + e < a.H) v[e >> 1] |= (int)((uint32_t)reinterpret_cast<const uint16_t*>(xr)[k + e] << (16 * (e & 1)));
    }
    return v;
  };
  auto x_put = [&](int n, v4i v) {
    const int p = (int)threadIdx.x + 256 * n;
    *reinterpret_cast<v4i*>(smem + x_at(p >> 2, p & 3)) = v;
  };
  const v4i x0 = x_piece(0), x1 = x_piece(1);
  int e = -1;
  for (int r = 0; r <= rank; ++r) e = lg.take(lane);
  if (e < 0) return;                                     // the whole workgroup
  // this wave's groups of 4 columns, g0 + kUpWaves * j, segment by segment
  const int g0 = kUpWaves * a.per * tile + wave, groups = (a.I + 3) / 4;
  const int items = max(0, min(a.per, (groups - g0 + kUpWaves - 1) / kUpWaves)) * segs;
  const uint8_t* w = a.w13 + e * a.st_w13;
  const uint8_t* s = a.s13 + e * a.st_s13;
  int asked = 0, ask_i = 4 * g0, ask_seg = 0;            // the next item to be asked for
  auto ask = [&](Block& blk) {
    if (asked == items) return;
    blk.ask<4>(0, w, a.ld_w13, s, a.ld_s13, ask_i, a.I - 1, 64 * ask_seg + lane, nb);
    blk.ask<4>(4, w, a.ld_w13, s, a.ld_s13, a.I + ask_i, 2 * a.I - 1, 64 * ask_seg + lane, nb);
    ++asked;
    if (++ask_seg == segs) {
      ask_seg = 0;
      ask_i += 4 * kUpWaves;
    }
  };
  Block b0, b1;
  ask(b0);
  ask(b1);
  x_put(0, x0);
  if (segs > 1) x_put(1, x1);
  for (int n = 2; n < segs; ++n) x_put(n, x_piece(n));
  __syncthreads();
  float acc[kRows] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  int i0 = 4 * g0, seg = 0;                              // the next item to be multiplied
  auto multiply = [&](Block& blk) {
    const int b = 64 * seg + lane;
    float x[32];
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const v4i v = lds16(x_at(b, q), 0);
#pragma unroll
      for (int d = 0; d < 4; ++d) {
        x[8 * q + 2 * d] = __uint_as_float((uint32_t)v[d] << 16);
        x[8 * q + 2 * d + 1] = __uint_as_float((uint32_t)v[d] & 0xFFFF0000u);
      }
    }
    blk.dot(x, b < nb, acc);
    ask(blk);
    if (++seg < segs) return;
    seg = 0;
    const float gate = sum_rows(acc, lane), up = __shfl_xor(gate, 32);
#pragma unroll
    for (int q = 0; q < kRows; ++q) acc[q] = 0.0f;
    const int i = i0 + (lane >> 3);
    i0 += 4 * kUpWaves;
    if (lane < 32 && (lane & 7) == 0) {                  // the group's piece is filled with zeros past I
      float* h = reinterpret_cast<float*>(a.h + slot * hidden_bytes(a.I)) + (i / kSeg) * kSeg + (i % 32 / 4) * 256 + (i % kSeg / 32) * 4;
      h[i & 3] = i < a.I ? silu(gate) * up : 0.0f;
    }
  };
#pragma unroll 1
  for (int n = 0; n < items; n += 2) {
    multiply(b0);
    if (n + 1 < items) multiply(b1);
  }
}

__global__ __launch_bounds__(64 * kDownWaves, 2) void k_moe_few_down(const MoeArgs a) {
  __shared__ float sums[2][kDownWaves][kRows];
  const int t = blockIdx.y;
  const int lane = threadIdx.x & 63, waves = blockDim.x / 64;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int nb = (a.I + 31) / 32, segs = (a.I + kSeg - 1) / kSeg;
  Logits<kKeys> lg;
  lg.load(a, t, lane);
  const float top = lg.top();
  float all = 0.0f;
  if (!a.renorm) {
#pragma unroll
    for (int q = 0; q < kKeys; ++q) all += 64 * q + lane < a.E ? expf(lg.l[q] - top) : 0.0f;
    all = wave_sum(all);
  }
  // lane r: the expert of rank r and exp(its logit - top)
  int mine = -1, kept = 0;
  for (int r = 0; r < a.k; ++r) {
    const int e = lg.take(lane);
    if (e < 0) break;
    if (lane == r) mine = e;
    ++kept;
  }
  const float p = mine >= 0 ? expf((a.logits + t * a.ld_logits)[mine] - top) : 0.0f;
  const float share = p / (a.renorm ? wave_sum(p) : all);
  // the wave's items: its units wave, wave + waves, ... of the workgroup's first row group, then of the next
  const int units = kept * segs;
  const int groups = (a.H + kRows - 1) / kRows, stride = kRows * (int)gridDim.x;
  const int own = (groups - (int)blockIdx.x + (int)gridDim.x - 1) / (int)gridDim.x;
  int ask_u = wave, ask_row = kRows * (int)blockIdx.x;   // the next item to be asked for
  auto ask = [&](Block& blk) {
    if (ask_u >= units || ask_row >= a.H) return;
    const int r = ask_u / segs, e = __builtin_amdgcn_readlane(mine, r);
    blk.ask<kRows>(0, a.w2 + e * a.st_w2, a.ld_w2, a.s2 + e * a.st_s2, a.ld_s2, ask_row, a.H - 1,
                   64 * (ask_u - r * segs) + lane, nb);
    ask_u += waves;
    if (ask_u >= units) {
      ask_u = wave;
      ask_row += stride;
    }
  };
  v4i hn[8];                                             // the lane's block of the next unit's h
  auto hidden = [&](int u) {
    const int r = u / segs, seg = u - r * segs;
    const uint8_t* h = a.h + (int64_t)(t * a.k + r) * hidden_bytes(a.I) + (int64_t)seg * (4 * kSeg);
    const int left = a.I - kSeg * seg - 32 * lane;
#pragma unroll
    for (int q = 0; q < 8; ++q) hn[q] = *reinterpret_cast<const v4i*>(h + (4 * q < left ? 1024u * q + 16u * lane : 0u));
  };
  Block next;
  ask(next);
  if (wave < units) hidden(wave);
  float acc[kRows] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
  const bool one = wave + waves >= units;                // a wave with one unit keeps its h
#pragma unroll 1
  for (int j = 0; j < own; ++j) {
#pragma unroll 1
    for (int u = wave; u < units; u += waves) {
      const int r = u / segs, seg = u - r * segs;
      const Block now = next;
      float x[32];
#pragma unroll
      for (int q = 0; q < 32; ++q) x[q] = __uint_as_float((uint32_t)hn[q >> 2][q & 3]);
      if (kSeg * (seg + 1) > a.I) {                      // what lies past I was not stored
#pragma unroll
        for (int q = 0; q < 32; ++q) x[q] = kSeg * seg + 32 * lane + q < a.I ? x[q] : 0.0f;
      }
      ask(next);
      if (!one) hidden(u + waves < units ? u + waves : wave);
      float dot[kRows] = {0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f, 0.0f};
      now.dot(x, 64 * seg + lane < nb, dot);
      const float sh = __uint_as_float((uint32_t)__builtin_amdgcn_readlane((int)__float_as_uint(share), r));
#pragma unroll
      for (int q = 0; q < kRows; ++q) acc[q] = __builtin_fmaf(sh, dot[q], acc[q]);
    }
    const float s = sum_rows(acc, lane);
#pragma unroll
    for (int q = 0; q < kRows; ++q) acc[q] = 0.0f;
    if ((lane & 7) == 0) sums[j & 1][wave][lane >> 3] = s;
    __syncthreads();                                     // the next group's sums go to the other half
    const int col = kRows * (int)blockIdx.x + stride * j + (int)threadIdx.x;
    if (threadIdx.x < kRows && col < a.H) {
      float y = 0.0f;
      for (int w = 0; w < waves; ++w) y += sums[j & 1][w][threadIdx.x];
      if (a.y_bf16)
        reinterpret_cast<uint16_t*>(a.y)[t * a.ld_y + col] = (uint16_t)f32_to_bf16_rne(y);
      else
        reinterpret_cast<float*>(a.y)[t * a.ld_y + col] = y;
    }
  }
}

}  // namespace few
}  // namespace

namespace {
namespace few {

// Column groups of a wave going up, with two workgroups a CU, as many as the registers allow.
int64_t up_per(int64_t T, int64_t I, int64_t k, int cus) {
  const int64_t tiles = (I + 4 * kUpWaves - 1) / (4 * kUpWaves), room = 2 * (int64_t)cus;
  return (T * k * tiles + room - 1) / room;
}

// Going down a CU has room for 8 waves.  A workgroup of w goes through `own` row groups, and each costs
// it its waves' units and half of one for adding them up: the cheapest w.
struct Down {
  int waves;
  int64_t own;
  double cost;
};

Down down_of(int64_t T, int64_t H, int64_t I, int64_t k, int cus) {
  const int64_t units = k * ((I + kSeg - 1) / kSeg), groups = (H + kRows - 1) / kRows;
  Down best{1, 0, 1e30};
  for (int w = 1; w <= kDownWaves && w <= units; ++w) {
    const int64_t room = ((int64_t)cus * (kDownWaves / w) + T - 1) / T, own = (groups + room - 1) / room;
    const double cost = own * ((units + w - 1) / w + 0.5);
    if (cost < best.cost) best = Down{w, own, cost};
  }
  return best;
}

}  // namespace few
}  // namespace

// Fits to runs on 256 CUs: 2.9 us for an item of 8 rows x 2048 elements going up, 3 us down.  Measured
// and estimated: up 13.9 and 9.8 us, down 9.3 and 7.5 (1 token, 4 of 64 experts of 4096 x 2048); 51 and
// 50, 32 and 30 (8 tokens of the same); 24.8 and 21, 22.1 and 22 (7 tokens, 6 of 60, 2000 x 1064).
double moe_few_us(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int cus) {
  if (H > 8 * few::kSeg || E > 64 * few::kKeys || k > 64) return 1e30;
  return 7 + 2.9 * (double)few::up_per(T, I, k, cus) * (double)((H + few::kSeg - 1) / few::kSeg) +
         3.0 * few::down_of(T, H, I, k, cus).cost;
}

int64_t moe_few_bytes(int64_t T, int64_t I, int64_t k) { return T * k * few::hidden_bytes(I); }

hipError_t launch_moe_few(const MoeArgs& args, hipStream_t st) {
  MoeArgs a = args;
  const int64_t tiles = (a.I + 4 * few::kUpWaves - 1) / (4 * few::kUpWaves), slots = (int64_t)a.T * a.k;
  const int cus = device_cu_count();
  a.per = (int)few::up_per(a.T, a.I, a.k, cus);
  a.tiles = (int)((tiles + a.per - 1) / a.per);
  if (slots * a.tiles > 0x7FFFFFFF) return hipErrorInvalidValue;
  const int segs = (a.H + few::kSeg - 1) / few::kSeg;
  hipLaunchKernelGGL(few::k_moe_few_up, dim3((unsigned)(slots * a.tiles)), dim3(64 * few::kUpWaves), 2 * few::kSeg * segs, st, a);
  const hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  const few::Down d = few::down_of(a.T, a.H, a.I, a.k, cus);
  const int64_t groups = (a.H + few::kRows - 1) / few::kRows;
  hipLaunchKernelGGL(few::k_moe_few_down, dim3((unsigned)((groups + d.own - 1) / d.own), (unsigned)a.T), dim3(64 * d.waves), 0, st,
                     a);
  return hipGetLastError();
}

}  // namespace mxq
