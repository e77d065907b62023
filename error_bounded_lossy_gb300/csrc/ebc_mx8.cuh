// ebc_mx8.cuh -- the 8-bit microscaled format (see include/ebc.h): a block's
// scale, a value's code, and back; and a row's values between memory and lanes.
#pragma once

#include <type_traits>

#include "ebc_types.cuh"

namespace ebc {

// The scale byte of a block with largest magnitude amax (its bits): e + 127 for
// the least e >= -127 with amax <= 448 * 2^e, 255 for a NaN or an infinity.
//   amax = m * 2^b, m in [1, 2):  amax <= 1.75 * 2^8 * 2^(b-8) exactly when m <= 7/4,
// so e is b - 8 or b - 7, read off the exponent and the fraction's top bits.
__device__ __forceinline__ uint32_t mx8_scale(uint32_t bits) {
  const uint32_t b = bits >> 23;
  if (b == 255u) return 255u;
  const int s = (int)b - 8 + ((bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return s < 0 ? 0u : (uint32_t)s;
}

// 2^-(s - 127), exact: s is at most 247 for a finite block.
__device__ __forceinline__ float mx8_inverse(uint32_t s) { return __uint_as_float((254u - s) << 23); }

// 2^(s - 127) (a subnormal for s = 0), NaN for 255.
__device__ __forceinline__ float mx8_unit(uint32_t s) {
  return s == 255u ? __uint_as_float(0x7FC00000u) : s == 0u ? __uint_as_float(0x00400000u) : __uint_as_float(s << 23);
}

// The codes of two values, `lo` in the low byte: to nearest, ties to even.
__device__ __forceinline__ uint32_t mx8_codes2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}

// The values of two codes (exact in a half).
__device__ __forceinline__ float2 mx8_values2(uint32_t codes) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"((uint16_t)codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&r));
}

// V consecutive values of a row (1, 2 or 8): as they are in memory, one access.
template <typename T, int V>
struct Values {
  static constexpr int kBytes = V * (int)sizeof(T), kWords = (kBytes + 3) / 4;
  union {
    uint32_t word[kWords];
    uint16_t half[2 * kWords];
    T e[V];
  };
  __device__ __forceinline__ Values() {}
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (kBytes == 32)
      asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3]), "=r"(word[4]), "=r"(word[5]),
                     "=r"(word[6]), "=r"(word[7])
                   : "l"(p));
    else if constexpr (kBytes == 16)
      asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                   : "=r"(word[0]), "=r"(word[1]), "=r"(word[2]), "=r"(word[3])
                   : "l"(p));
    else if constexpr (kBytes == 8)
      asm volatile("ld.global.v2.b32 {%0, %1}, [%2];" : "=r"(word[0]), "=r"(word[1]) : "l"(p));
    else if constexpr (kBytes == 4)
      asm volatile("ld.global.b32 %0, [%1];" : "=r"(word[0]) : "l"(p));
    else
      asm volatile("ld.global.b16 %0, [%1];" : "=h"(half[0]) : "l"(p));
  }
  __device__ __forceinline__ void store(T* p) const {
    if constexpr (kBytes == 32)
      asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(word[0]), "r"(word[1]),
                   "r"(word[2]), "r"(word[3]), "r"(word[4]), "r"(word[5]), "r"(word[6]), "r"(word[7]), "l"(p)
                   : "memory");
    else if constexpr (kBytes == 16)
      asm volatile("st.global.v4.b32 [%4], {%0, %1, %2, %3};" ::"r"(word[0]), "r"(word[1]), "r"(word[2]),
                   "r"(word[3]), "l"(p)
                   : "memory");
    else if constexpr (kBytes == 8)
      asm volatile("st.global.v2.b32 [%2], {%0, %1};" ::"r"(word[0]), "r"(word[1]), "l"(p) : "memory");
    else if constexpr (kBytes == 4)
      asm volatile("st.global.b32 [%1], %0;" ::"r"(word[0]), "l"(p) : "memory");
    else
      asm volatile("st.global.b16 [%1], %0;" ::"h"(half[0]), "l"(p) : "memory");
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int k = 0; k < kWords; ++k) word[k] = 0u;
  }
  // As fp32, and from fp32 to nearest: two 16-bit values at a time, which is half
  // of the instructions that one at a time takes, and less.
  __device__ __forceinline__ void get(float (&f)[V]) const {
    if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
      for (int k = 0; k < V; ++k) f[k] = to_f32(e[k]);
    } else {
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          f[2 * k] = __uint_as_float(word[k] << 16);
          f[2 * k + 1] = __uint_as_float(word[k] & 0xFFFF0000u);
        } else {
          const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&word[k]));
          f[2 * k] = v.x;
          f[2 * k + 1] = v.y;
        }
      }
    }
  }
  __device__ __forceinline__ void set(const float (&f)[V]) {
    if constexpr (sizeof(T) == 4 || V == 1) {
#pragma unroll
      for (int k = 0; k < V; ++k) e[k] = from_f32<T>(f[k]);
    } else {
#pragma unroll
      for (int k = 0; k < V / 2; ++k) {
        if constexpr (std::is_same<T, __nv_bfloat16>::value) {
          const __nv_bfloat162 v = __floats2bfloat162_rn(f[2 * k], f[2 * k + 1]);
          word[k] = *reinterpret_cast<const uint32_t*>(&v);
        } else {
          const __half2 v = __floats2half2_rn(f[2 * k], f[2 * k + 1]);
          word[k] = *reinterpret_cast<const uint32_t*>(&v);
        }
      }
    }
  }
};

// Values that one access takes: 8 where every address given (pointers and row
// strides in bytes, or'ed together) is a multiple of 8 values, else 2 or 1.
inline int row_values(uintptr_t addresses, int elem) {
  return addresses % (uintptr_t)(8 * elem) == 0 ? 8 : addresses % (uintptr_t)(2 * elem) == 0 ? 2 : 1;
}

// A block's largest magnitude (its bits; of a NaN, all of them but the sign), of
// the 32 / V lanes that hold it.
template <int V>
__device__ __forceinline__ uint32_t mx8_block_max(const float (&f)[V]) {
  float top = fabsf(f[0]);
#pragma unroll
  for (int k = 1; k < V; ++k) asm("max.NaN.f32 %0, %0, %1;" : "+f"(top) : "f"(fabsf(f[k])));
  // (magnitudes order as their bits do, and a NaN's are above an infinity's)
  if constexpr (V == 1) {
    return __reduce_max_sync(0xffffffffu, __float_as_uint(top));
  } else {
    uint32_t bits = __float_as_uint(top);
#pragma unroll
    for (int off = 1; off < 32 / V; off <<= 1) bits = max(bits, __shfl_xor_sync(0xffffffffu, bits, off));
    return bits & 0x7FFFFFFFu;
  }
}

// The lane's codes of a block with that scale, to `codes` (aligned to V).
template <int V>
__device__ __forceinline__ void mx8_store(const float (&f)[V], uint32_t scale, uint8_t* codes) {
  const float inv = mx8_inverse(scale);   // (of 255: not used)
  const uint32_t keep = scale == 255u ? 0u : ~0u;
  auto code2 = [&](float lo, float hi) { return mx8_codes2(lo * inv, hi * inv) & keep; };
  if constexpr (V == 8) {
    const uint32_t a = mx8_codes2(f[0] * inv, f[1] * inv) | mx8_codes2(f[2] * inv, f[3] * inv) << 16;
    const uint32_t b = mx8_codes2(f[4] * inv, f[5] * inv) | mx8_codes2(f[6] * inv, f[7] * inv) << 16;
    *reinterpret_cast<uint2*>(codes) = make_uint2(a & keep, b & keep);
  } else if constexpr (V == 2) {
    *reinterpret_cast<uint16_t*>(codes) = (uint16_t)code2(f[0], f[1]);
  } else {
    *codes = (uint8_t)code2(f[0], 0.f);
  }
}

}  // namespace ebc
