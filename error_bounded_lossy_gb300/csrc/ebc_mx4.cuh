// ebc_mx4.cuh -- the 4-bit microscaled format (see include/ebc.h): a block's
// scale, a value's code, and back.
#pragma once

#include "ebc_types.cuh"

namespace ebc {

// The scale byte of a block with largest magnitude amax: e + 127 for the least
// e >= -127 with amax <= 6 * 2^e, 255 for a NaN or an infinity.
//   amax = m * 2^b, m in [1, 2):  amax <= 6 * 2^(b-2) exactly when m <= 3/2,
// so e is b - 2 or b - 1, read off the exponent and the fraction's top bits.
__device__ __forceinline__ uint32_t mx4_scale(float amax) {
  const uint32_t bits = __float_as_uint(amax), b = bits >> 23;
  if (b == 255u) return 255u;
  const int s = (int)b - 2 + ((bits & 0x7FFFFFu) > 0x400000u ? 1 : 0);
  return s < 0 ? 0u : (uint32_t)s;
}

// 2^-(s - 127), exact: s is at most 253 for a finite block.
__device__ __forceinline__ float mx4_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// 2^(s - 127) (a subnormal for s = 0), NaN for 255.
__device__ __forceinline__ float mx4_unit(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7FC00000u) : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// The codes of two values, `lo` in the low four bits: to nearest, ties to the
// even code.
__device__ __forceinline__ uint32_t mx4_pair(float lo, float hi) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.rn.satfinite.e2m1x2.f32 t, %1, %2;\n cvt.u32.u8 %0, t;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The values of the two codes in the low byte of `pair`, as halves (exact).
__device__ __forceinline__ __half2 mx4_values(uint32_t pair) {
  uint32_t r;
  asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(r) : "r"(pair));
  return *reinterpret_cast<__half2*>(&r);
}

}  // namespace ebc
