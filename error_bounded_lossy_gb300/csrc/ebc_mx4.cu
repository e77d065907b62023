// ebc_mx4.cu -- rows to 4-bit microscaled values and back, alone and on the
// way into the experts' sending buffer.  See include/ebc.h for the format.
#include "ebc_mx4.cuh"

using namespace ebc;

namespace {

constexpr int kMxWarps = 8;
constexpr int kSpan = 512;   // values of a warp's piece: one 16-byte group of scales
// a / b; most often in 32 bits, a fifth of the instructions
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return a <= UINT32_MAX ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

constexpr int kLane = 8;     // consecutive values of a lane; a block is four lanes

// Eight consecutive values of a row (zeros past its end) as they are in
// memory: 16-byte loads where the row is aligned for them, else one by one.
template <typename T>
struct Eight {
  static constexpr int kWords = kLane * (int)sizeof(T) / 4;
  union {
    uint4 raw[kWords / 4];
    uint32_t word[kWords];
    T e[kLane];
  };
  __device__ __forceinline__ Eight() {}
};
template <typename T, bool kAligned>
__device__ __forceinline__ void load8(const T* row, int64_t h, int64_t width, Eight<T>* v) {
  if (kAligned && h + kLane <= width) {
#pragma unroll
    for (int i = 0; i < Eight<T>::kWords / 4; ++i) v->raw[i] = reinterpret_cast<const uint4*>(row + h)[i];
  } else {
#pragma unroll
    for (int k = 0; k < kLane; ++k) v->e[k] = h + k < width ? row[h + k] : from_f32<T>(0.f);
  }
}

// The largest magnitude of a block, four lanes' values.  Magnitudes order as
// their bits do, and a NaN's bits are above an infinity's, so neither gets
// lost; 16-bit types are compared two at a time.
__device__ __forceinline__ float block_max(const Eight<float>& v) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kLane; ++k) top = max(top, v.word[k] & 0x7FFFFFFFu);
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
  return __uint_as_float(top);
}
template <typename T>
__device__ __forceinline__ float block_max(const Eight<T>& v) {
  uint32_t top = 0;
#pragma unroll
  for (int k = 0; k < kLane / 2; ++k) top = __vmaxu2(top, v.word[k] & 0x7FFF7FFFu);
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = __vmaxu2(top, __shfl_xor_sync(0xffffffffu, top, 2));
  const uint16_t one = (uint16_t)max(top & 0xFFFFu, top >> 16);
  return to_f32(*reinterpret_cast<const T*>(&one));
}

// The lane's eight codes and its block's scale byte.
template <typename T>
__device__ __forceinline__ uint32_t encode8(const Eight<T>& v, uint32_t* scale) {
  const uint32_t s = mx4_scale(block_max(v));
  *scale = s;
  if (s == 255u) return 0u;
  const float inv = mx4_inverse(s);
  uint32_t c = 0;
#pragma unroll
  for (int k = 0; k < kLane; k += 2) c |= mx4_pair(to_f32(v.e[k]) * inv, to_f32(v.e[k + 1]) * inv) << (4 * k);
  return c;
}

// A warp takes 512 values of a row (two times eight a lane), so that it owns a
// whole 16-byte group of scales.  With kRoute each token's codes go to the
// rows of its choices: quantized once, written `top` times, and rows past the
// last expert's are zero.  Bound by bandwidth: 16 or 32 bits read and 4.25
// written a value.
template <typename T, bool kAligned, bool kRoute>
__global__ void __launch_bounds__(32 * kMxWarps) k_mx4_quantize(const T* __restrict__ x, int64_t ld, int64_t rows,
                                                                int64_t width, int top,
                                                                const int32_t* __restrict__ place,
                                                                const int32_t* __restrict__ offsets, int E,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales, Glob* glob) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t spans = (width + kSpan - 1) / kSpan;
  const int64_t code_bytes = EBC_MX4_CODE_BYTES(width), scale_bytes = spans * 16, blocks = (width + 31) / 32;
  const int64_t n = rows * top;
  int64_t live = n;
  if (kRoute) {
    live = offsets[E];
    live = live < 0 ? 0 : live < n ? live : n;
  }
  const int64_t units = (rows + (n - live)) * spans;
  for (int64_t u = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kMxWarps) {
    const int64_t t = divide(u, spans), span = u - t * spans;
    uint32_t c[2] = {0u, 0u}, s[2] = {0u, 0u};
    if (!kRoute || t < rows) {
      Eight<T> v[2];
#pragma unroll
      for (int i = 0; i < 2; ++i)
        load8<T, kAligned>(x + t * ld, span * kSpan + i * 256 + lane * kLane, width, &v[i]);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        c[i] = encode8(v[i], &s[i]);
        if (span * 16 + i * 8 + lane / 4 >= blocks) s[i] = 0u;
      }
    }
    auto store = [&](int64_t r) {
      uint8_t* cr = codes + r * code_bytes;
      uint8_t* sr = scales + r * scale_bytes + span * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int64_t at = span * 256 + i * 128 + lane * 4;
        if (at < code_bytes) *reinterpret_cast<uint32_t*>(cr + at) = c[i];
        if ((lane & 3) == 0) sr[i * 8 + lane / 4] = (uint8_t)s[i];
      }
    };
    if (!kRoute) {
      store(t);
    } else if (t < rows) {
      for (int j = 0; j < top; ++j) {
        const int32_t p = place[t * top + j];
        if (p >= n && lane == 0) record_error(glob, EBC_ERR_INVALID_ARG);
        if (p >= 0 && p < n) store(p);
      }
    } else {
      store(live + (t - rows));
    }
  }
}

// A lane takes eight codes.  Bound by the bandwidth of the writes.
template <typename T, bool kAligned>
__global__ void __launch_bounds__(32 * kMxWarps) k_mx4_dequantize(const uint8_t* __restrict__ codes,
                                                                  const uint8_t* __restrict__ scales, int64_t rows,
                                                                  int64_t width, T* __restrict__ x) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t spans = (width + kSpan - 1) / kSpan;
  const int64_t code_bytes = EBC_MX4_CODE_BYTES(width), scale_bytes = spans * 16;
  for (int64_t u = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5); u < rows * spans;
       u += (int64_t)gridDim.x * kMxWarps) {
    const int64_t t = divide(u, spans), span = u - t * spans;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int64_t h = span * kSpan + i * 256 + lane * kLane;
      if (h >= width) continue;
      const uint32_t c = *reinterpret_cast<const uint32_t*>(codes + t * code_bytes + h / 2);
      const float unit = mx4_unit(scales[t * scale_bytes + h / 32]);
      float v[kLane];
#pragma unroll
      for (int k = 0; k < kLane; k += 2) {
        const float2 f = __half22float2(mx4_values((c >> (4 * k)) & 0xFFu));
        v[k] = f.x * unit;
        v[k + 1] = f.y * unit;
      }
      T* dst = x + t * width + h;
      if (kAligned && h + kLane <= width) {
        constexpr int kN = 16 / (int)sizeof(T);
#pragma unroll
        for (int q = 0; q < kLane / kN; ++q) {
          Vec<T, 16> o;
#pragma unroll
          for (int k = 0; k < kN; ++k) o.e[k] = from_f32<T>(v[q * kN + k]);
          *reinterpret_cast<uint4*>(dst + q * kN) = o.raw;
        }
      } else {
#pragma unroll
        for (int k = 0; k < kLane; ++k)
          if (h + k < width) dst[k] = from_f32<T>(v[k]);
      }
    }
  }
}

unsigned mx_grid(int64_t units, int nsm) {
  const int64_t want = (units + kMxWarps - 1) / kMxWarps, most = (int64_t)nsm * 8 * 8;
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

bool mx_rows_ok(int64_t rows, int64_t width) {
  return rows >= 0 && rows <= INT32_MAX && width >= 1 && width <= (1 << 24);
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

template <typename T, bool kRoute>
cudaError_t quantize_t(const CallView& v, const void* x, int64_t ld, int64_t rows, int64_t width, int top,
                       const int32_t* place, const int32_t* offsets, int E, uint8_t* codes, uint8_t* scales,
                       cudaStream_t st) {
  const bool al = aligned(x, 16) && (ld * (int64_t)sizeof(T)) % 16 == 0;
  const dim3 grid(mx_grid(rows * ((width + kSpan - 1) / kSpan), v.nsm)), block(32 * kMxWarps);
  const char* name = kRoute ? "k_mx4_dispatch" : "k_mx4_quantize";
  return al ? launch_named(v, name, st, k_mx4_quantize<T, true, kRoute>, grid, block, 0, 1, (const T*)x, ld, rows,
                           width, top, place, offsets, E, codes, scales, v.glob)
            : launch_named(v, name, st, k_mx4_quantize<T, false, kRoute>, grid, block, 0, 1, (const T*)x, ld, rows,
                           width, top, place, offsets, E, codes, scales, v.glob);
}

template <bool kRoute>
int quantize_any(ebc_ctx* ctx, const void* x, int64_t ld, int type, int64_t rows, int64_t width, int top,
                 const int32_t* place, const int32_t* offsets, int E, uint8_t* codes, uint8_t* scales,
                 void* stream) {
  const int b = type_bytes(type);
  if (!ctx || !b || !mx_rows_ok(rows, width) || ld < width || ld > ((int64_t)1 << 40)) return EBC_ERR_INVALID_ARG;
  if (kRoute && (top < 1 || top > EBC_MAX_EXPERTS || rows > (int64_t)INT32_MAX / top || E < 1 ||
                 E > EBC_MAX_EXPERTS || !offsets || !aligned(offsets, 4) || (rows > 0 && (!place || !aligned(place, 4)))))
    return EBC_ERR_INVALID_ARG;
  if (rows > 0 && (!x || !aligned(x, b) || !codes || !aligned(codes, 16) || !scales || !aligned(scales, 16)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || rows == 0) return rc;
  cudaError_t e;
  if (type == EBC_F32)
    e = quantize_t<float, kRoute>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
  else if (type == EBC_BF16)
    e = quantize_t<__nv_bfloat16, kRoute>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
  else
    e = quantize_t<__half, kRoute>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
  return cuda_code(e);
}

template <typename T>
cudaError_t dequantize_t(const CallView& v, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t width,
                         void* x, cudaStream_t st) {
  const bool al = aligned(x, 16) && (width * (int64_t)sizeof(T)) % 16 == 0;
  const dim3 grid(mx_grid(rows * ((width + kSpan - 1) / kSpan), v.nsm)), block(32 * kMxWarps);
  return al ? launch_named(v, "k_mx4_dequantize", st, k_mx4_dequantize<T, true>, grid, block, 0, 1, codes, scales,
                           rows, width, (T*)x)
            : launch_named(v, "k_mx4_dequantize", st, k_mx4_dequantize<T, false>, grid, block, 0, 1, codes, scales,
                           rows, width, (T*)x);
}

}  // namespace

extern "C" {

int ebc_mx4_quantize(ebc_ctx* ctx, const void* d_x, int64_t ld_x, int type, int64_t rows, int64_t width,
                     uint8_t* d_codes, uint8_t* d_scales, void* stream) {
  return quantize_any<false>(ctx, d_x, ld_x, type, rows, width, 1, nullptr, nullptr, 1, d_codes, d_scales, stream);
}

int ebc_moe_dispatch_mx4(ebc_ctx* ctx, const void* d_x, int64_t ld_x, int type, int64_t tokens, int top,
                         int64_t width, const int32_t* d_place, const int32_t* d_offsets, int n_experts,
                         uint8_t* d_codes, uint8_t* d_scales, void* stream) {
  return quantize_any<true>(ctx, d_x, ld_x, type, tokens, width, top, d_place, d_offsets, n_experts, d_codes,
                            d_scales, stream);
}

int ebc_mx4_dequantize(ebc_ctx* ctx, const uint8_t* d_codes, const uint8_t* d_scales, int64_t rows, int64_t width,
                       int type, void* d_xhat, void* stream) {
  const int b = type_bytes(type);
  if (!ctx || !b || !mx_rows_ok(rows, width)) return EBC_ERR_INVALID_ARG;
  if (rows > 0 && (!d_codes || !aligned(d_codes, 16) || !d_scales || !aligned(d_scales, 16) || !d_xhat ||
                   !aligned(d_xhat, b)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || rows == 0) return rc;
  if (type == EBC_F32) return cuda_code(dequantize_t<float>(v, d_codes, d_scales, rows, width, d_xhat, st));
  if (type == EBC_BF16) return cuda_code(dequantize_t<__nv_bfloat16>(v, d_codes, d_scales, rows, width, d_xhat, st));
  return cuda_code(dequantize_t<__half>(v, d_codes, d_scales, rows, width, d_xhat, st));
}

}  // extern "C"
