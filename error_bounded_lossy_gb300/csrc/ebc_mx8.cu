// ebc_mx8.cu -- rows to 8-bit microscaled values and back.  See include/ebc.h
// for the format.
#include "ebc_mx8.cuh"

using namespace ebc;

namespace {

constexpr int kWarps = 8;

// a / b; most often in 32 bits, a fifth of the instructions
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return a <= UINT32_MAX ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Rows as one run of vectors of V values, filled up to whole blocks, so that
// short rows leave no lane idle: vector v of row t is number t * each + v.
struct Rows {
  int64_t rows, width, ld;
  int each;          // vectors of a row
  uint32_t scale_bytes;
};

// The row (past the unit's first) and the place in it of vector v, counted from
// that row's start.  Mostly a unit ends before the second row does.
template <int kPieces>
__device__ __forceinline__ void place(const Rows& r, uint32_t v, uint32_t* row, uint32_t* vec) {
  const uint32_t each = (uint32_t)r.each;
  *row = each >= 32u * kPieces ? (v >= each ? 1u : 0u) : v / each;
  *vec = v - *row * each;
}

// A warp takes kPieces runs of 32 vectors, all in flight at once; a block is
// 32 / V lanes.  The lanes of a row's last block also fill up its scales.
// 16 or 32 bits are read and 8.25 written a value: bound by bandwidth.
template <typename T, int V, int kPieces>
__global__ void __launch_bounds__(32 * kWarps) k_mx8_quantize(const T* x, Rows r, uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  pdl_enter();
  constexpr int kLanes = 32 / V;   // of a block
  const int lane = threadIdx.x & 31, at = lane & (kLanes - 1);
  const int64_t code_bytes = (int64_t)r.each * V;
  const int64_t units = (r.rows * r.each + 32 * kPieces - 1) / (32 * kPieces);
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
    const int64_t first = u * (32 * kPieces), t0 = divide(first, r.each);
    const uint32_t v0 = (uint32_t)(first - t0 * r.each) + lane;
    Values<T, V> in[kPieces];
    uint32_t row[kPieces], vec[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      place<kPieces>(r, v0 + 32 * i, &row[i], &vec[i]);
      const int64_t t = t0 + row[i], left = t < r.rows ? r.width - (int64_t)vec[i] * V : 0;
      const T* p = x + t * r.ld + (int64_t)vec[i] * V;
      if (left >= V) {
        in[i].load(p);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k) in[i].e[k] = k < left ? p[k] : from_f32<T>(0.f);
      }
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float f[V];
      in[i].get(f);
      const uint32_t s = mx8_scale(mx8_block_max<V>(f));
      const int64_t t = t0 + row[i];
      if (t >= r.rows) continue;
      mx8_store<V>(f, s, codes + t * code_bytes + (int64_t)vec[i] * V);
      uint8_t* sr = scales + t * r.scale_bytes;
      const uint32_t block = vec[i] / kLanes;
      if (at == 0) sr[block] = (uint8_t)s;
      if (block == (uint32_t)r.each / kLanes - 1)
        for (uint32_t b = block + 1 + at; b < r.scale_bytes; b += kLanes) sr[b] = 0;
    }
  }
}

// The way back, laid out the same (vectors of a row's values, no filling).
template <typename T, int V, int kPieces>
__global__ void __launch_bounds__(32 * kWarps) k_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, Rows r,
                                                                T* __restrict__ x) {
  pdl_enter();
  const int lane = threadIdx.x & 31;
  const int64_t code_bytes = (r.width + 31) / 32 * 32;
  const int64_t units = (r.rows * r.each + 32 * kPieces - 1) / (32 * kPieces);
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
    const int64_t first = u * (32 * kPieces), t0 = divide(first, r.each);
    const uint32_t v0 = (uint32_t)(first - t0 * r.each) + lane;
    uint2 c[kPieces];
    uint32_t s[kPieces], row[kPieces], vec[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      place<kPieces>(r, v0 + 32 * i, &row[i], &vec[i]);
      const int64_t t = t0 + row[i];
      if (t >= r.rows) continue;
      const uint8_t* p = codes + t * code_bytes + (int64_t)vec[i] * V;
      c[i].y = 0u;
      if constexpr (V == 8)
        c[i] = *reinterpret_cast<const uint2*>(p);
      else if constexpr (V == 2)
        c[i].x = *reinterpret_cast<const uint16_t*>(p);
      else
        c[i].x = *p;
      s[i] = scales[t * r.scale_bytes + vec[i] / (32 / V)];
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int64_t t = t0 + row[i];
      if (t >= r.rows) continue;
      const float unit = mx8_unit(s[i]);
      Values<T, V> out;
      float f[V];
#pragma unroll
      for (int k = 0; k < V; k += 2) {
        const float2 v = mx8_values2((k < 4 ? c[i].x : c[i].y) >> (8 * (k & 3)));
        f[k] = v.x * unit;
        if constexpr (V > 1) f[k + 1] = v.y * unit;
      }
      out.set(f);
      const int64_t left = r.width - (int64_t)vec[i] * V;
      T* p = x + t * r.width + (int64_t)vec[i] * V;
      if (left >= V) {
        out.store(p);
      } else {
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (k < left) p[k] = out.e[k];
      }
    }
  }
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

bool shape_ok(int64_t rows, int64_t width) {
  return rows >= 0 && rows <= INT32_MAX && width >= 1 && width <= (1 << 24);
}

// CTAs for the rows' vectors, at most two full turns of the machine; the
// kernels loop beyond that.
unsigned grid(int64_t vectors, int pieces, int nsm) {
  const int64_t want = (vectors + 32 * pieces * kWarps - 1) / (32 * pieces * kWarps), most = (int64_t)nsm * 8 * 2;
  return (unsigned)(want < most ? want : most);
}

// Runs of a warp: as many (up to four) as leave 24 warps for each SM.
int pieces(int64_t vectors, int nsm) {
  int p = 4;
  while (p > 1 && vectors < (int64_t)nsm * 24 * 32 * p) p /= 2;
  return p;
}

template <typename F>
cudaError_t with_pieces(int p, F&& f) {
  if (p == 4) return f(std::integral_constant<int, 4>{});
  if (p == 2) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}
template <typename T, typename F>
cudaError_t with_values(int v, F&& f) {
  if (v == 8) return f(std::integral_constant<int, 8>{});
  if (v == 2) return f(std::integral_constant<int, 2>{});
  return f(std::integral_constant<int, 1>{});
}

template <typename T>
cudaError_t quantize_t(const CallView& v, const T* x, int64_t ld, int64_t rows, int64_t width, uint8_t* codes,
                       uint8_t* scales, cudaStream_t st) {
  return with_values<T>(row_values((uintptr_t)x | (uintptr_t)(ld * (int64_t)sizeof(T)), sizeof(T)), [&](auto tv) {
    constexpr int V = tv();
    const Rows r{rows, width, ld, (int)((width + 31) / 32 * (32 / V)), (uint32_t)EBC_MX8_SCALE_BYTES(width)};
    return with_pieces(pieces(rows * r.each, v.nsm), [&](auto tp) {
      return launch_named(v, "k_mx8_quantize", st, k_mx8_quantize<T, V, tp()>,
                          dim3(grid(rows * r.each, tp(), v.nsm)), dim3(32 * kWarps), 0, 1, x, r, codes, scales);
    });
  });
}

template <typename T>
cudaError_t dequantize_t(const CallView& v, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t width,
                         T* x, cudaStream_t st) {
  return with_values<T>(row_values((uintptr_t)x | (uintptr_t)(width * (int64_t)sizeof(T)), sizeof(T)), [&](auto tv) {
    constexpr int V = tv();
    const Rows r{rows, width, width, (int)((width + V - 1) / V), (uint32_t)EBC_MX8_SCALE_BYTES(width)};
    return with_pieces(pieces(rows * r.each, v.nsm), [&](auto tp) {
      return launch_named(v, "k_mx8_dequantize", st, k_mx8_dequantize<T, V, tp()>,
                          dim3(grid(rows * r.each, tp(), v.nsm)), dim3(32 * kWarps), 0, 1, codes, scales, r, x);
    });
  });
}

}  // namespace

extern "C" {

int ebc_mx8_quantize(ebc_ctx* ctx, const void* d_x, int64_t ld_x, int type, int64_t rows, int64_t width,
                     uint8_t* d_codes, uint8_t* d_scales, void* stream) {
  const int b = type_bytes(type);
  if (!ctx || !b || !shape_ok(rows, width) || ld_x < width || ld_x > ((int64_t)1 << 40)) return EBC_ERR_INVALID_ARG;
  if (rows > 0 && (!d_x || !aligned(d_x, b) || !d_codes || !aligned(d_codes, 16) || !d_scales || !aligned(d_scales, 16)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || rows == 0) return rc;
  if (type == EBC_F32) return cuda_code(quantize_t(v, (const float*)d_x, ld_x, rows, width, d_codes, d_scales, st));
  if (type == EBC_BF16)
    return cuda_code(quantize_t(v, (const __nv_bfloat16*)d_x, ld_x, rows, width, d_codes, d_scales, st));
  return cuda_code(quantize_t(v, (const __half*)d_x, ld_x, rows, width, d_codes, d_scales, st));
}

int ebc_mx8_dequantize(ebc_ctx* ctx, const uint8_t* d_codes, const uint8_t* d_scales, int64_t rows, int64_t width,
                       int type, void* d_xhat, void* stream) {
  const int b = type_bytes(type);
  if (!ctx || !b || !shape_ok(rows, width)) return EBC_ERR_INVALID_ARG;
  if (rows > 0 && (!d_codes || !aligned(d_codes, 16) || !d_scales || !aligned(d_scales, 16) || !d_xhat ||
                   !aligned(d_xhat, b)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || rows == 0) return rc;
  if (type == EBC_F32) return cuda_code(dequantize_t(v, d_codes, d_scales, rows, width, (float*)d_xhat, st));
  if (type == EBC_BF16) return cuda_code(dequantize_t(v, d_codes, d_scales, rows, width, (__nv_bfloat16*)d_xhat, st));
  return cuda_code(dequantize_t(v, d_codes, d_scales, rows, width, (__half*)d_xhat, st));
}

}  // extern "C"
