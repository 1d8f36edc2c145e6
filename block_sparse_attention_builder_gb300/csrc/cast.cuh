// Value casts shared by the kernels that write and read the paged caches:
// the 16-bit types, unscaled e4m3 and the NVFP4 groups (E2M1 codes with one
// E4M3 scale per 16 elements).
#pragma once
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <cstdint>

namespace mxsa {

__device__ __forceinline__ float to_f32(uint16_t bits, int bf16) {
  return bf16 ? __uint_as_float((uint32_t)bits << 16) : __half2float(__ushort_as_half(bits));
}

// e4m3 code of x, rounded to nearest even and saturating at 448 (the largest
// finite value, so saturating equals clamping first); a NaN gives a NaN code
__device__ __forceinline__ uint32_t e4m3_code2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// e4m3 codes of two source values (raw 16-bit words b0, b1), b0's in the
// low byte (no NaN among them)
__device__ __forceinline__ uint32_t e4m3x2(uint16_t b0, uint16_t b1, int bf16) {
  return e4m3_code2(to_f32(b0, bf16), to_f32(b1, bf16));
}

// the same, for a 16-bit word that may be a NaN: the code takes the NaN's
// sign from the source bits (the fp16 -> f32 conversion does not keep it)
__device__ __forceinline__ uint32_t e4m3_nan_aware(uint16_t b, int bf16) {
  const bool nan = (b & 0x7FFFu) > (bf16 ? 0x7F80u : 0x7C00u);
  return nan ? ((b & 0x8000u) ? 0xFFu : 0x7Fu) : (e4m3x2(b, 0, bf16) & 0xFFu);
}

// any NaN among the eight 16-bit values of s
__device__ __forceinline__ bool any_nan(const uint4& s, int bf16) {
  const uint32_t thr = bf16 ? 0x7F807F80u : 0x7C007C00u;
  const uint32_t w[4] = {s.x, s.y, s.z, s.w};
  uint32_t hit = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) hit |= __vcmpgtu2(w[i] & 0x7FFF7FFFu, thr);
  return hit != 0;
}

// one 16-byte source chunk s (8 values) to its destination: 8 e4m3 bytes or
// the 16 bytes themselves
__device__ __forceinline__ void put_chunk(const uint4& s, uint8_t* dst, long long dst_elem, int fp8, int bf16) {
  if (fp8) {
    uint32_t o[2];
    if (!any_nan(s, bf16)) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t x = i ? s.z : s.x, y = i ? s.w : s.y;
        o[i] = e4m3x2((uint16_t)(x & 0xFFFFu), (uint16_t)(x >> 16), bf16) |
               (e4m3x2((uint16_t)(y & 0xFFFFu), (uint16_t)(y >> 16), bf16) << 16);
      }
    } else {
      const uint32_t w4[4] = {s.x, s.y, s.z, s.w};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        o[i] = 0;
#pragma unroll
        for (int b = 0; b < 4; ++b)
          o[i] |= e4m3_nan_aware((uint16_t)(w4[2 * i + b / 2] >> (16 * (b & 1))), bf16) << (8 * b);
      }
    }
    *reinterpret_cast<uint2*>(dst + dst_elem) = make_uint2(o[0], o[1]);
  } else {
    *reinterpret_cast<uint4*>(dst + 2 * dst_elem) = s;
  }
}

// the values of two e4m3 codes (low byte first) as packed halves, exactly
__device__ __forceinline__ uint32_t e4m3x2_to_f16x2(uint16_t codes) {
  uint32_t h2;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h2) : "h"(codes));
  return h2;
}

// E2M1 code of y: the comparisons put each tie on the even magnitude index
// (0.25 -> 0, 0.75 and 1.25 -> 1.0, 1.75 and 2.5 -> 2, 3.5 and 5 -> 4)
__device__ __forceinline__ uint32_t e2m1_code(float y) {
  const uint32_t sign = (__float_as_uint(y) >> 31) << 3;
  const float a = fabsf(y);
  uint32_t i;
  if (a <= 0.25f) i = 0;
  else if (a < 0.75f) i = 1;
  else if (a <= 1.25f) i = 2;
  else if (a < 1.75f) i = 3;
  else if (a <= 2.5f) i = 4;
  else if (a < 3.5f) i = 5;
  else if (a <= 5.0f) i = 6;
  else i = 7;
  return sign | i;
}

// the e4m3 scale of a group whose largest magnitude is amax, and its value
__device__ __forceinline__ uint32_t nvfp4_scale(float amax, float* value) {
  const uint32_t sc = e4m3_code2(__fdiv_rn(amax, 6.f), 0.f) & 0xFFu;
  *value = __half2float(__ushort_as_half((uint16_t)(e4m3x2_to_f16x2((uint16_t)sc) & 0xFFFFu)));
  return sc;
}

// code of one element under the scale value sd
__device__ __forceinline__ uint32_t nvfp4_code(float x, float sd) {
  return (sd == 0.f || isnan(x)) ? 0u : e2m1_code(__fdiv_rn(x, sd));
}

// y, which has x's sign or is a zero, with x's sign
__device__ __forceinline__ float with_sign(float y, float x) {
  return __uint_as_float(__float_as_uint(y) | (__float_as_uint(x) & 0x80000000u));
}

// codes of eight elements of a group under the scale value sd, the first in
// the low bits.  Quotients by the reciprocal and one residual step, correctly
// rounded for a correctly rounded reciprocal (Markstein 1990, theorem 8), so
// the same as nvfp4_code's but for the sign of a zero, which is x's; a quotient
// too small for an exact residual has code 0 either way.  Groups with infinities or NaN, and a scale of
// 0, take nvfp4_code.
__device__ __forceinline__ uint32_t nvfp4_codes8(const float* x, float sd) {
  const float s = ((x[0] + x[1]) + (x[2] + x[3])) + ((x[4] + x[5]) + (x[6] + x[7]));
  uint32_t codes = 0;
  if (sd != 0.f && fabsf(s) < INFINITY) {
    const float r = __frcp_rn(sd);
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float q0 = x[i] * r, q1 = x[i + 1] * r;
      const float y0 = with_sign(fmaf(fmaf(-q0, sd, x[i]), r, q0), x[i]);
      const float y1 = with_sign(fmaf(fmaf(-q1, sd, x[i + 1]), r, q1), x[i + 1]);
      uint32_t c;
      asm("{\n\t.reg .b8 b;\n\tcvt.rn.satfinite.e2m1x2.f32 b, %1, %2;\n\tcvt.u32.u8 %0, b;\n\t}"
          : "=r"(c)
          : "f"(y1), "f"(y0));
      codes |= c << (4 * i);
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) codes |= nvfp4_code(x[i], sd) << (4 * i);
  }
  return codes;
}

}  // namespace mxsa
