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

// The codes of eight values, the first in the low four bits: to nearest, ties
// to the even code.
__device__ __forceinline__ uint32_t mx4_codes(const float (&v)[8]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n"
      " cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n"
      " cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n"
      " mov.b32 %0, {a, b, c, d};\n}\n"
      : "=r"(r)
      : "f"(v[0]), "f"(v[1]), "f"(v[2]), "f"(v[3]), "f"(v[4]), "f"(v[5]), "f"(v[6]), "f"(v[7]));
  return r;
}

// The values of eight codes, as four pairs of halves (exact).
__device__ __forceinline__ void mx4_values(uint32_t codes, __half2 (&v)[4]) {
  uint32_t r[4];
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}\n"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
      : "r"(codes));
#pragma unroll
  for (int i = 0; i < 4; ++i) v[i] = *reinterpret_cast<__half2*>(&r[i]);
}

}  // namespace ebc
