// The block-scaled 8-bit format: e4m3 codes with one power-of-two scale per group of 128.
//
// A group's scale is 2^e with the least e for which max|x| <= 448 * 2^e (448 is the largest e4m3
// value), held as the e8m0 byte e + 127.  Dividing an fp32 value by 2^e is exact (or falls far
// below e4m3's least value), so a code is its value rounded once, to nearest even.
#pragma once

#include <cstdint>

namespace tp {

constexpr int kFp8Group = 128;

// e8m0 byte of a group from the bits of its largest |x| (sign cleared, as fp32).  Integer order
// of those bits is the order of the values with infinity and then NaN on top, so a maximum taken
// over the bits keeps a NaN.  A group that holds either gets 255, the format's NaN.
__device__ __forceinline__ uint32_t e8m0_of_amax(uint32_t abs_bits) {
  if (abs_bits >= 0x7F800000u) return 255u;
  if (abs_bits == 0u) return 127u;
  // |x| = 1.f * 2^(E-127), 448 = 1.75 * 2^8 (1.75 has the mantissa field 0x600000); a subnormal
  // fp32 (E = 0) clamps to the format's least scale, 2^-127.
  const int e = static_cast<int>(abs_bits >> 23) - 8 + ((abs_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return static_cast<uint32_t>(max(e, 0));
}

// 2^-e of an e8m0 byte (NaN for 255, so that every code of such a group becomes NaN).
__device__ __forceinline__ float e8m0_inverse(uint32_t byte) {
  return __uint_as_float(byte == 255u ? 0x7FFFFFFFu : (254u - byte) << 23);
}

// Two fp32 values as e4m3 codes, `lo` in the low byte (nearest even; NaN stays NaN).
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) {
  return e4m3x2(a, b) | (e4m3x2(c, d) << 16);
}

__device__ __forceinline__ uint32_t abs_bits(float v) { return __float_as_uint(v) & 0x7FFFFFFFu; }

// The larger magnitude of two values, NaN if either is, with a sign that means nothing.
__device__ __forceinline__ float max_abs(float a, float b) {
  float r;
  asm("max.NaN.xorsign.abs.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}

}  // namespace tp
