// fp4_mma.hpp -- the skinny product of MXFP4 weights on gfx950: a workgroup multiplies 16 * NT
// rows of W [N][K] with 16 * MT rows of X, its waves splitting K.
//
// The unit of work is 128 elements of K.  Both operands go from memory to the matrix cores
// in registers: lane l = 16 g + i loads the 16 bytes of MX block 4u + g of W row i, one block
// under one scale byte.
//   X in bf16: the block's 32 codes are decoded with their scale to bf16 (exact) and feed four
//     v_mfma_f32_16x16x32_bf16 (exact products, FP32 sums); MFMA j holds the block's elements
//     8j .. 8j+7, for which the lane reads 16 bytes of X.  Any assignment of k to (MFMA, lane
//     group, element) is right as long as both operands share it.
//   X in MXFP4: v_mfma_scale_f32_16x16x128_f8f6f4 takes codes and scale bytes as they are.
//     E2M1 products are multiples of 1/4 up to 36, so the sums inside a block are exact, and
//     the block sums combine with their scales in FP32 (measured within 4e-8 of sum |x w|).
// W is the A operand, so lane (i, g) ends up with rows 4g .. 4g+3 of W (output columns) of X
// row i.
#pragma once
#include "codec4.hpp"
#include "gemm_common.hpp"

namespace mxq {
namespace {

typedef float v4f __attribute__((ext_vector_type(4)));

constexpr int kUnit = 128;             // elements of K per unit: 4 blocks

enum : int { kXBf16 = 0, kXFp4 = 1 };

__device__ __forceinline__ v4i load16(const uint8_t* p) {   // any alignment
  v4i v;
  __builtin_memcpy(&v, p, 16);
  return v;
}

// Keep the first n (0 .. 32) of the 32 codes in four dwords.
__device__ __forceinline__ v4i keep_codes(v4i v, int n) {
#pragma unroll
  for (int d = 0; d < 4; ++d) {
    const int r = n - 8 * d;
    const uint32_t m = r >= 8 ? 0xFFFFFFFFu : r <= 0 ? 0u : (1u << (4 * r)) - 1u;
    v[d] = (int)((uint32_t)v[d] & m);
  }
  return v;
}

// One unit's operands of a lane.
template <int XT, int MT, int NT>
struct Unit {
  v4i w[NT];
  uint32_t ws[NT];
  v4i x[MT][XT == kXBf16 ? 4 : 1];
  uint32_t xs[MT];
};

// The lane's operand rows.  w / ws: first row of the workgroup (uniform), wo / so the lane's
// row offsets in it (block 4u + g adds 64 u + 16 g and 4u + g); x / xs: the lane's X rows.
template <int MT, int NT>
struct Rows {
  const uint8_t* w;
  const uint8_t* ws;
  uint32_t wo[NT], so[NT];
  const uint8_t* x[MT];
  const uint8_t* xs[MT];
};

template <int XT, int MT, int NT>
__device__ __forceinline__ void load_unit(Unit<XT, MT, NT>& t, const Rows<MT, NT>& r, int u, int g) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    t.w[n] = *reinterpret_cast<const v4i*>(r.w + (r.wo[n] + 64u * (uint32_t)u));
    t.ws[n] = r.ws[r.so[n] + 4u * (uint32_t)u];
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (XT == kXBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) t.x[m][XT == kXBf16 ? j : 0] = load16(r.x[m] + 256 * (int64_t)u + 64 * g + 16 * j);
    } else {
      t.x[m][0] = *reinterpret_cast<const v4i*>(r.x[m] + 64 * (int64_t)u + 16 * g);
      t.xs[m] = r.xs[m][4 * (int64_t)u + g];
    }
  }
}

// The last unit of a K that is no multiple of 128: blocks past the end are zero under scale 1,
// elements at k >= K are zero in both operands.
template <int XT, int MT, int NT>
__device__ __forceinline__ void load_unit_tail(Unit<XT, MT, NT>& t, const Rows<MT, NT>& r, int u, int g, int K) {
  const int left = K - kUnit * u - 32 * g;             // elements of the lane's block
  const v4i zero = {0, 0, 0, 0};
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    t.w[n] = zero;
    t.ws[n] = 127u;
    if (left > 0) {
      t.w[n] = keep_codes(*reinterpret_cast<const v4i*>(r.w + (r.wo[n] + 64u * (uint32_t)u)), left);
      t.ws[n] = r.ws[r.so[n] + 4u * (uint32_t)u];
    }
  }
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    if (XT == kXBf16) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v4i v = zero;
        const uint16_t* p = reinterpret_cast<const uint16_t*>(r.x[m] + 256 * (int64_t)u + 64 * g + 16 * j);
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (8 * j + e < left) v[e >> 1] |= (int)((uint32_t)p[e] << (16 * (e & 1)));
        t.x[m][XT == kXBf16 ? j : 0] = v;
      }
    } else {
      t.x[m][0] = zero;
      t.xs[m] = 127u;
      if (left > 0) {
        t.x[m][0] = keep_codes(*reinterpret_cast<const v4i*>(r.x[m] + 64 * (int64_t)u + 16 * g), left);
        t.xs[m] = r.xs[m][4 * (int64_t)u + g];
      }
    }
  }
}

template <int XT, int MT, int NT>
__device__ __forceinline__ void mma_unit(const Unit<XT, MT, NT>& t, v4f acc[MT][NT]) {
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    if (XT == kXBf16) {
      const float s = e8m0_to_f32(t.ws[n]);
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t d[4];
        fp4::decode8_bf16((uint32_t)t.w[n][j], s, d);
        const v4i dv = {(int)d[0], (int)d[1], (int)d[2], (int)d[3]};
#pragma unroll
        for (int m = 0; m < MT; ++m)
          acc[m][n] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(
              __builtin_bit_cast(v8bf, dv), __builtin_bit_cast(v8bf, t.x[m][XT == kXBf16 ? j : 0]), acc[m][n], 0, 0, 0);
      }
    } else {
      const v8i a = {t.w[n][0], t.w[n][1], t.w[n][2], t.w[n][3], 0, 0, 0, 0};
#pragma unroll
      for (int m = 0; m < MT; ++m) {
        const v8i b = {t.x[m][0][0], t.x[m][0][1], t.x[m][0][2], t.x[m][0][3], 0, 0, 0, 0};
        acc[m][n] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, b, acc[m][n], 4, 4, 0, (int)t.ws[n], 0,
                                                                     (int)t.xs[m]);
      }
    }
  }
}

// Sums of the wave's units u0, u0 + step, ... of K, with D units of loads in flight.
template <int XT, int MT, int NT, int D>
__device__ __forceinline__ void sum_units(const Rows<MT, NT>& r, int u0, int step, int g, int K, v4f acc[MT][NT]) {
  const int full = K / kUnit;
  Unit<XT, MT, NT> t[D];
#pragma unroll
  for (int d = 0; d < D; ++d)
    if (u0 + d * step < full) load_unit(t[d], r, u0 + d * step, g);
  int u = u0;
  while (u < full) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (u < full) {
        mma_unit<XT, MT, NT>(t[d], acc);
        if (u + D * step < full) load_unit(t[d], r, u + D * step, g);
      }
      u += step;
    }
  }
  if (K % kUnit != 0 && full % step == u0) {           // the partial unit is number `full`
    load_unit_tail(t[0], r, full, g, K);
    mma_unit<XT, MT, NT>(t[0], acc);
  }
}

// The waves' sums side by side in LDS: wave w's value of X row m, W row n is at
// [w][m][n], rows of 16 * NT + 4 floats (the pad spreads the 16 rows that a store covers).
template <int NT>
constexpr int part_row() { return 16 * NT + 4; }
template <int MT, int NT>
constexpr int part_wave() { return 16 * MT * part_row<NT>(); }

template <int MT, int NT>
__device__ __forceinline__ void store_part(float* part, int wave, int lane, const v4f acc[MT][NT]) {
  const int i = lane & 15, g = lane >> 4;
#pragma unroll
  for (int m = 0; m < MT; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n)
      *reinterpret_cast<v4f*>(part + wave * part_wave<MT, NT>() + (16 * m + i) * part_row<NT>() + 16 * n + 4 * g) =
          acc[m][n];
}

// Sum over `waves` waves, in wave order, of X row m, W rows n .. n+3.
template <int MT, int NT>
__device__ __forceinline__ v4f sum_part(const float* part, int waves, int m, int n) {
  v4f s = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int w = 0; w < waves; ++w)
    s += *reinterpret_cast<const v4f*>(part + w * part_wave<MT, NT>() + m * part_row<NT>() + n);
  return s;
}

}  // namespace
}  // namespace mxq
