// Rounding to the storage formats (sm_100a), shared by the cache write sides.
#pragma once

#include "common.cuh"

namespace lidx {

// smallest e in [-127, 127] with amax <= top * 2^e (amax finite, > 0), for a
// format whose largest value is top = m * 2^ex_top with m in [1, 2), given as
// m's mantissa bits: amax = m' * 2^x needs e = x - ex_top when m' <= m, else
// one more (a subnormal amax is below top * 2^-127 for both formats).
// E4M3: 448 = 1.75 * 2^8; E2M1: 6 = 1.5 * 2^2.
__device__ __forceinline__ int block_exponent(float amax, uint32_t mantissa, int ex_top) {
  const uint32_t u = __float_as_uint(amax);
  return max(-127, static_cast<int>(u >> 23) - 127 - ex_top + ((u & 0x7FFFFFu) > mantissa ? 1 : 0));
}
__device__ __forceinline__ int block_exponent_e4m3(float amax) { return block_exponent(amax, 0x600000u, 8); }
__device__ __forceinline__ int block_exponent_e2m1(float amax) { return block_exponent(amax, 0x400000u, 2); }

// 2^-e, exactly, for e in [-127, 126] (the exponents of finite magnitudes)
__device__ __forceinline__ float inverse_scale(int e) { return __uint_as_float(static_cast<uint32_t>(127 - e) << 23); }

__device__ __forceinline__ uint32_t e4m3x2(float hi, float lo) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// E4M3 code of v already divided by its block scale: NaN -> 0x7F, |v| > 448
// saturates, else the nearest code (ties to even).
__device__ __forceinline__ float e4m3_prep(float v) {
  return fabsf(v) > 448.f ? copysignf(448.f, v) : v;  // NaN compares false and stays NaN
}

__device__ __forceinline__ uint32_t pack4_e4m3(const float *v) {
  uint32_t c[4];
#pragma unroll
  for (int i = 0; i < 4; i++) c[i] = is_nan_bits(v[i]) ? 0x7Fu : 0u;
  const uint32_t lo = e4m3x2(e4m3_prep(v[1]), e4m3_prep(v[0]));
  const uint32_t hi = e4m3x2(e4m3_prep(v[3]), e4m3_prep(v[2]));
  uint32_t r = lo | (hi << 16);
#pragma unroll
  for (int i = 0; i < 4; i++)
    if (c[i]) r = (r & ~(0xFFu << (8 * i))) | (0x7Fu << (8 * i));
  return r;
}

// Eight E2M1 codes of finite v already divided by its block scale, v[0] in the
// low nibble: the nearest value (ties to the even code), |v| > 6 saturating.
__device__ __forceinline__ uint32_t pack8_e2m1_finite(const float *s) {
  uint32_t r;
  asm("{\n"
      " .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n"
      " cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n"
      " cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n"
      "}\n"
      : "=r"(r)
      : "f"(s[0]), "f"(s[1]), "f"(s[2]), "f"(s[3]), "f"(s[4]), "f"(s[5]), "f"(s[6]), "f"(s[7]));
  return r;
}

// The same for any v: NaN as +6, infinities saturating.
__device__ __forceinline__ uint32_t pack8_e2m1(const float *v) {
  float s[8];
#pragma unroll
  for (int i = 0; i < 8; i++) s[i] = is_nan_bits(v[i]) ? 6.f : v[i];
  return pack8_e2m1_finite(s);
}

// Four E4M3 codes of v with |v| <= 448.
__device__ __forceinline__ uint32_t pack4_e4m3_in_range(const float *v) {
  return e4m3x2(v[1], v[0]) | (e4m3x2(v[3], v[2]) << 16);
}

// bf16 bits of x, nearest even; NaN keeps its payload's top bits, quieted
__device__ __forceinline__ uint32_t bf16_bits(float x) {
  const uint32_t u = __float_as_uint(x);
  if (is_nan_bits(x)) return (u >> 16) | 0x40u;
  return __bfloat16_as_ushort(__float2bfloat16_rn(x));
}

// pack8_bf16 of values that are not NaN
__device__ __forceinline__ uint4 pack8_bf16_numbers(const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) {
    const __nv_bfloat162 two = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    w[i] = *reinterpret_cast<const uint32_t *>(&two);
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

__device__ __forceinline__ uint4 pack8_bf16(const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; i++) w[i] = bf16_bits(v[2 * i]) | (bf16_bits(v[2 * i + 1]) << 16);
  return make_uint4(w[0], w[1], w[2], w[3]);
}

}  // namespace lidx
