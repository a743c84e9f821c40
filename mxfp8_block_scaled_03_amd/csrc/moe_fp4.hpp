// moe_fp4.hpp -- what the kernels of the expert layer share: their arguments, the order of
// logits, and the layout of the hidden values.
#pragma once
#include <math.h>

#include "fp4_stream.hpp"

namespace mxq {

constexpr uint32_t kMasked = 0x007FFFFFu;   // order key of -inf

struct MoeArgs {
  int T, H, I, E, k, renorm;
  int slots, by_token;                 // by_token: slot = (token, rank), else slot = expert
  int mt_cap;                          // 16-row tiles that a slot's part of h holds
  int tiles, per;                      // column tiles of a launch; column groups of a wave (moe_fp4_few.hip)
  const uint8_t* x;
  int64_t ld_x;                        // bytes
  bool x_pieces;                       // X rows are whole 16-byte pieces
  bool s13_words, s2_words;            // scale rows are whole 4-byte words
  bool s13_pieces, s2_pieces;          // and 16-byte aligned
  const float* logits;
  int64_t ld_logits;
  const uint8_t *w13, *s13, *w2, *s2;
  int64_t ld_w13, st_w13, ld_s13, st_s13, ld_w2, st_w2, ld_s2, st_s2;   // rows and experts, bytes
  int* chosen;                         // [T][k]: expert, or -1
  float* share;                        // [T][k]
  int16_t* rank;                       // [E][T]: rank of the expert for the token, or -1
  uint8_t* h;                          // [slots][mt_cap][chunks][4 steps][planes][4][64][16 bytes]
  int parts;                           // K ranges of the down product
  float* part;                         // [T * k][parts][H]
  void* y;
  int64_t ld_y;
  int y_bf16;
};

namespace {

// Order key of a logit: greater for greater values, equal for -0 and +0, NaN above +inf.
__device__ __forceinline__ uint32_t order_key(float l) {
  if (l != l) return 0xFFFFFFFFu;
  const uint32_t b = __float_as_uint(l + 0.0f);
  return b ^ (b >> 31 ? 0xFFFFFFFFu : 0x80000000u);
}

template <int CTRL>
__device__ __forceinline__ uint32_t max_dpp(uint32_t v) {
  const uint32_t o = (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, true);
  return v > o ? v : o;
}

// The greatest of the wave's values: within rows of 16 lanes, then across them; lane 63 has it.
__device__ __forceinline__ uint32_t wave_umax(uint32_t v) {
  v = max_dpp<0x111>(v);                     // row_shr 1, 2, 4, 8
  v = max_dpp<0x112>(v);
  v = max_dpp<0x114>(v);
  v = max_dpp<0x118>(v);
  v = max_dpp<0x142>(v);                     // row_bcast 15, 31
  v = max_dpp<0x143>(v);
  return (uint32_t)__builtin_amdgcn_readlane((int)v, 63);
}

__device__ __forceinline__ float wave_sum(float v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// The logits of a token, lane l those of experts l, l + 64, ..., at most KEYS.
template <int KEYS>
struct Logits {
  float l[KEYS];
  uint32_t key[KEYS];                        // 0 past the last and once taken

  __device__ __forceinline__ void load(const MoeArgs& a, int t, int lane) {
    const float* row = a.logits + t * a.ld_logits;
#pragma unroll
    for (int q = 0; q < KEYS; ++q) {
      const int j = 64 * q + lane;
      l[q] = j < a.E ? row[j] : -__builtin_inff();
    }
#pragma unroll
    for (int q = 0; q < KEYS; ++q) key[q] = 64 * q + lane < a.E ? order_key(l[q]) : 0u;
  }

  // The greatest of them, NaN if one is.
  __device__ __forceinline__ float top() const {
    float v = -__builtin_inff();
    bool nan = false;
#pragma unroll
    for (int q = 0; q < KEYS; ++q) {
      v = fmaxf(v, l[q]);
      nan |= l[q] != l[q];
    }
#pragma unroll
    for (int d = 32; d > 0; d >>= 1) v = fmaxf(v, __shfl_xor(v, d));
    return __any(nan) ? __builtin_nanf("") : v;
  }

  // Takes the greatest logit's expert, the lowest of equals; -1 where only masked ones are left.
  __device__ __forceinline__ int take(int lane) {
    uint32_t m = 0;
#pragma unroll
    for (int q = 0; q < KEYS; ++q) m = m > key[q] ? m : key[q];
    m = wave_umax(m);
    if (m <= kMasked) return -1;
    int e = -1;
#pragma unroll
    for (int q = KEYS - 1; q >= 0; --q) {
      const uint64_t b = __ballot(key[q] == m);
      if (b != 0) e = 64 * q + __ffsll((unsigned long long)b) - 1;
    }
#pragma unroll
    for (int q = 0; q < KEYS; ++q)
      if (e == 64 * q + lane) key[q] = 0u;
    return e;
  }
};

// The hidden values go from one product to the next in the second one's fragment order, as bf16 terms
// that the matrix cores take as they are, a plane of 16 bytes per 8 elements each (XWide): two terms,
// 16 bits, where y is bf16 (its own rounding is 2^-8), or three, all 24 bits, where it is fp32 (cut
// from fp32 in the down product instead, once per wave and use, they took 34 us against 27: 7 tokens,
// 60 experts of 2000 x 1064).  Bytes of 16 rows x one chunk:
constexpr int hidden_chunk(int kind) { return 16384 * kind; }

// Byte offset in a 16-row tile of h of the 16 bytes of plane 0 that hold row m's elements k .. k+7.
template <int KIND>
__device__ __forceinline__ int64_t h_offset(int m, int k) {
  const int c = k / kChunk, b = (k % kChunk) / 32;       // block b = 4 g + u of the chunk
  return ((int64_t)(4 * c + b % 4) * (4 * KIND) + (k % 32) / 8) * 1024 + (16 * (b / 4) + m) * 16;
}

// Four hidden values, elements 4 half .. 4 half + 3 of the eight at `to` (plane 0).  The terms are
// rounded to nearest, so each is exact to 2^-9 of the one before.  The first one is finite, at most
// bf16's greatest, so that what FP32 holds beyond it is not lost: the rest, an infinity or a NaN too, is for
// the next; an infinity has no further term.
template <int KIND>
__device__ __forceinline__ void store_hidden(uint8_t* to, int half, const float v[4]) {
  const float most = __uint_as_float(0x7F7F7FFFu);       // the last that rounds to bf16's greatest
  uint32_t t[KIND][4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    float rest = v[e];
#pragma unroll
    for (int p = 0; p < KIND; ++p) {
      t[p][e] = f32_to_bf16_rne(p == 0 ? __builtin_amdgcn_fmed3f(rest, -most, most) : rest);
      rest = p > 0 && (t[p][e] & 0x7F80u) == 0x7F80u ? 0.0f : rest - __uint_as_float(t[p][e] << 16);
    }
  }
#pragma unroll
  for (int p = 0; p < KIND; ++p)
    *reinterpret_cast<uint2*>(to + 4096 * p + 8 * half) = make_uint2(t[p][0] | (t[p][1] << 16), t[p][2] | (t[p][3] << 16));
}

// Share times the gated value of one hidden element, SiLU in fp32.
__device__ __forceinline__ float gated(float share, float gate, float up) { return share * (silu(gate) * up); }

}  // namespace

// The kernels of many workgroups' worth of weights (moe_fp4_wide.hip): rows of X in whole 16-byte
// pieces and H a multiple of 8, scale rows 16-byte aligned.  up fills h, down fills part.
template <int KIND>
hipError_t launch_moe_up_wide(const MoeArgs& a, hipStream_t st);
template <int KIND>
hipError_t launch_moe_down_wide(const MoeArgs& a, hipStream_t st);

// The layer where hardly an expert has two tokens (moe_fp4_few.hip): from the logits to y, with h as its
// only workspace.  The estimate of its time is without bound where it does not take the sizes.
double moe_few_us(int64_t T, int64_t H, int64_t I, int64_t E, int64_t k, int cus);
int64_t moe_few_bytes(int64_t T, int64_t I, int64_t k);
hipError_t launch_moe_few(const MoeArgs& a, hipStream_t st);

}  // namespace mxq
