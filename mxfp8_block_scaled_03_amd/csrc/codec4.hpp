// codec4.hpp -- device-side MXFP4 codec for gfx950: E8M0 scale selection for E2M1 elements,
// round-to-nearest-even and stochastic E2M1 encode, decode through the scaled conversions.
//
// MXFP4 is the OCP Microscaling Formats (MX) Specification v1.0 format of 4-bit elements:
// 32 consecutive values along the contraction axis share one E8M0 byte s (2^(s-127), 255 is
// NaN); an element is E2M1: sign, two exponent bits (bias 1), one mantissa bit, so its
// magnitudes are 0, 0.5, 1, 1.5, 2, 3, 4, 6 (codes 0..7), with no infinity and no NaN.  Two
// codes share a byte, the even element in the low half.
//
// The scaled conversions were checked on gfx950 against the definition:
// v_cvt_scalef32_pk_fp4_{bf16,f32} gives RNE(x / scale) saturated to +-6 (every bf16 pattern
// at scales 2^-126 .. 2^127; a million fp32 values and all midpoints), and
// v_cvt_scalef32_pk_{bf16,f32}_fp4 gives code * 2^(s-127) rounded once for all 16 codes x 256
// scale bytes, NaN for byte 255.
#pragma once
#include "codec.hpp"
#include "mxblock.hpp"

namespace mxq {
namespace fp4 {

using mxblock::Chunk;
using mxblock::chunk_abs_max;
using mxblock::value_bits;

// Scale byte from the fp32 bit pattern of a block's amax.  6 = 1.5 * 2^2, so with amax =
// 1.f * 2^E the smallest e with amax <= 6 * 2^e is E - 2 while f <= 0.5, else E - 1; the OCP
// rule is E - 2 always.  Clamped at e = -127; zero -> 127 (S = 1); Inf or NaN -> 255.
template <int R>
__device__ __forceinline__ uint32_t scale_byte(uint32_t abits) {
  if (abits >= 0x7F800000u) return 255u;
  if (abits == 0u) return 127u;
  const int eb = (int)(abits >> 23);
  const int byte = eb - 2 + (R == kRuleCeil && (abits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return eb == 0 || byte < 0 ? 0u : (uint32_t)byte;
}

// Scale 2^(sb-127) of a finite scale byte as a normal fp32 (byte 0 has none) and its inverse.
__device__ __forceinline__ float scale_of(uint32_t sb) { return __uint_as_float(sb << 23); }
__device__ __forceinline__ float inv_scale_of(uint32_t sb) { return __uint_as_float((254u - sb) << 23); }

__device__ __forceinline__ uint32_t cvt2_f32(uint32_t old, float a, float b, float s, int byte) {
  switch (byte) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, s, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, s, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, s, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(old, a, b, s, 3);
  }
}

__device__ __forceinline__ uint32_t cvt2_bf16(uint32_t old, uint32_t w, float s, int byte) {
  typedef __bf16 v2 __attribute__((ext_vector_type(2)));
  const v2 x = __builtin_bit_cast(v2, w);
  switch (byte) {
    case 0: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, x, s, 0);
    case 1: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, x, s, 1);
    case 2: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, x, s, 2);
    default: return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(old, x, s, 3);
  }
}

// RNE codes of 8 values (fp32 bit patterns) under scale byte sb: one dword.  Byte 0
// (S = 2^-127, not a normal fp32) converts x * 2^127, which is exact for blocks that small,
// at scale 1; byte 255 (a NaN/Inf block) writes code 7 throughout.
__device__ __forceinline__ uint32_t encode8_f32(const uint32_t v[8], uint32_t sb) {
  if (sb == 255u) return 0x77777777u;
  const float s = sb == 0u ? 1.0f : scale_of(sb);
  const float m = sb == 0u ? 0x1p127f : 1.0f;
  uint32_t d = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) d = cvt2_f32(d, __uint_as_float(v[2 * i]) * m, __uint_as_float(v[2 * i + 1]) * m, s, i);
  return d;
}

template <int SRC_BF16>
__device__ __forceinline__ uint32_t encode8(const Chunk<SRC_BF16>& c, uint32_t sb) {
  if (SRC_BF16 && sb - 1u < 254u) {
    uint32_t d = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) d = cvt2_bf16(d, c.w[i], scale_of(sb), i);
    return d;
  }
  uint32_t v[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = value_bits<SRC_BF16>(c, i);
  return encode8_f32(v, sb);
}

// Stochastically rounded code of the value with fp32 pattern vb under a finite scale byte
// (inv = 2^(127 - sb)) and the 24-bit random integer r, given as the word w whose top 24 bits it is:
// between the neighbours l <= |a| < u, up iff r < 2^24 * (|a| - l) / (u - l).  With |a| = m * 2^x,
// 1 <= m < 2, the step is 2^(max(x, 0) - 1), so q = |a| / step is exact, floor(q) + 2 max(x, 0) is
// the lower code, and the fraction of q times 2^32 and r * 2^8 are exact too: the comparison decides
// exactly.  |a| can underflow fp32 only where the threshold is below 1: there any positive
// number decides alike, so a nonzero value is kept from becoming 0 (min(|v|, 2^-126) is 0 for
// zero alone).  The ceil rule keeps |a| <= 6.
__device__ __forceinline__ uint32_t encode_sr(uint32_t vb, float inv, uint32_t w) {
  const float v = __builtin_fabsf(__uint_as_float(vb));
  const float a = __builtin_fmaxf(v * inv, __builtin_fminf(v, 0x1p-126f));
  const int x1 = max(__builtin_amdgcn_frexp_expf(a), 1);               // max(x, 0) + 1
  const float q = __builtin_amdgcn_ldexpf(a, 2 - x1);
  const uint32_t up = (float)(w & 0xFFFFFF00u) < __builtin_amdgcn_fractf(q) * 0x1p32f ? 1u : 0u;
  return ((uint32_t)q + (uint32_t)(2 * x1 - 2) + up) | ((vb >> 28) & 8u);
}

// The random words of the 32 elements of a block, as mxblock::block_random24 before its shift; the
// three-operand xor is one instruction.
__device__ __forceinline__ void block_random(uint64_t block, uint64_t seed, uint32_t r[32]) {
#pragma unroll
  for (int g = 0; g < 8; ++g) {
    const uint64_t ctr = block * 8u + (uint64_t)g;
    uint32_t c[4] = {(uint32_t)ctr, (uint32_t)(ctr >> 32), 0u, 0u};
    uint32_t k0 = (uint32_t)seed, k1 = (uint32_t)(seed >> 32);
#pragma unroll
    for (int i = 0; i < 10; ++i) {
      const uint64_t p0 = (uint64_t)c[0] * 0xD2511F53u, p1 = (uint64_t)c[2] * 0xCD9E8D57u;
      c[0] = (uint32_t)__builtin_amdgcn_bitop3_b32((int)(p1 >> 32), (int)c[1], (int)k0, 0x96);
      c[1] = (uint32_t)p1;
      c[2] = (uint32_t)__builtin_amdgcn_bitop3_b32((int)(p0 >> 32), (int)c[3], (int)k1, 0x96);
      c[3] = (uint32_t)p0;
      k0 += 0x9E3779B9u;
      k1 += 0xBB67AE85u;
    }
#pragma unroll
    for (int w = 0; w < 4; ++w) r[4 * g + w] = c[w];
  }
}

// Eight codes of a dword times the scale s = e8m0_to_f32(byte), as eight bf16 values in four
// dwords: the RNE of the exact product, which is exact for scale bytes 0 .. 252 (6 * 2^125 is
// bf16's largest binade; 0.5 * 2^-127 a bf16 subnormal); bytes 253 and 254 can overflow to Inf,
// byte 255 gives NaN.
__device__ __forceinline__ void decode8_bf16(uint32_t w, float s, uint32_t out[4]) {
  out[0] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 0));
  out[1] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 1));
  out[2] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 2));
  out[3] = __builtin_bit_cast(uint32_t, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(w, s, 3));
}

__device__ __forceinline__ void decode4_f32(uint32_t w16, float s, float out[4]) {
  const auto a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w16, s, 0);
  const auto b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w16, s, 1);
  out[0] = a[0];
  out[1] = a[1];
  out[2] = b[0];
  out[3] = b[1];
}

}  // namespace fp4
}  // namespace mxq
