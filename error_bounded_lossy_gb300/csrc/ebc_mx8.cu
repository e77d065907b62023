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

// Rows as one run of vectors of eight values, filled up to whole blocks, so that
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

// A warp's 32 vectors of eight values between memory and its lanes.  kV = 8: rows
// whose vectors are aligned, one access a lane.  Other rows go through the warp's
// piece of shared memory in accesses of kV values, the lanes next to each other,
// where the vectors are of one row (they mostly are); else a lane takes its values
// one by one, which touches as many sectors as there are lanes.
template <typename T, int kV>
struct Piece {
  static constexpr int kSteps = 8 / kV;
  static constexpr int kStage = kV == 8 ? 1 : 256;   // values
  // p: the lane's vector; left: the row's values from there on (not above 0: none)
  static __device__ __forceinline__ void load(const T* p, int left, uint32_t row, T* stage, int lane,
                                              Values<T, 8>* v) {
    if constexpr (kV == 8) {
      if (left >= 8) {
        v->load(p);
        return;
      }
    } else {
      if (__all_sync(0xffffffffu, row == __shfl_sync(0xffffffffu, row, 0))) {
        const T* q = p - lane * 8;
        const int left0 = left + lane * 8;
        Values<T, kV> r[kSteps];
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int at = (i * 32 + lane) * kV;
          if (at < left0)
            r[i].load(q + at);
          else
            r[i].zero();
        }
        __syncwarp();   // the last piece has been taken
#pragma unroll
        for (int i = 0; i < kSteps; ++i) put(stage + (i * 32 + lane) * kV, r[i]);
        __syncwarp();
#pragma unroll
        for (int k = 0; k < Values<T, 8>::kWords; k += 4) {
          const uint4 w = reinterpret_cast<const uint4*>(stage + lane * 8)[k / 4];
          v->word[k] = w.x;
          v->word[k + 1] = w.y;
          v->word[k + 2] = w.z;
          v->word[k + 3] = w.w;
        }
        return;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) v->e[k] = k < left ? p[k] : from_f32<T>(0.f);
  }
  static __device__ __forceinline__ void store(T* p, int64_t left, uint32_t row, T* stage, int lane,
                                               const Values<T, 8>& v) {
    if constexpr (kV == 8) {
      if (left >= 8) {
        v.store(p);
        return;
      }
    } else {
      if (__all_sync(0xffffffffu, row == __shfl_sync(0xffffffffu, row, 0))) {
        T* q = p - lane * 8;
        const int64_t left0 = left + lane * 8;
        __syncwarp();
#pragma unroll
        for (int k = 0; k < Values<T, 8>::kWords; k += 4)
          reinterpret_cast<uint4*>(stage + lane * 8)[k / 4] =
              make_uint4(v.word[k], v.word[k + 1], v.word[k + 2], v.word[k + 3]);
        __syncwarp();
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          const int at = (i * 32 + lane) * kV;
          if (at < left0) {
            Values<T, kV> r;
            get(stage + at, &r);
            r.store(q + at);
          }
        }
        return;
      }
    }
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k < left) p[k] = v.e[k];
  }
  static __device__ __forceinline__ void put(T* at, const Values<T, kV>& r) {
    if constexpr (kV == 1)
      *at = r.e[0];
    else if constexpr (sizeof(T) == 2)
      *reinterpret_cast<uint32_t*>(at) = r.word[0];
    else
      *reinterpret_cast<uint2*>(at) = make_uint2(r.word[0], r.word[1]);
  }
  static __device__ __forceinline__ void get(const T* at, Values<T, kV>* r) {
    if constexpr (kV == 1) {
      r->e[0] = *at;
    } else if constexpr (sizeof(T) == 2) {
      r->word[0] = *reinterpret_cast<const uint32_t*>(at);
    } else {
      const uint2 w = *reinterpret_cast<const uint2*>(at);
      r->word[0] = w.x;
      r->word[1] = w.y;
    }
  }
};

// A warp takes kPieces runs of 32 vectors, all in flight at once; a block is
// four lanes.  The lanes of a row's last block also fill up its scales.
// 16 or 32 bits are read and 8.25 written a value: bound by bandwidth, for 16-bit
// types by issue as much.  [16384, 4096] bf16 36.6 us (5.6 TB/s), [8192, 3328] fp32
// 21.4 (6.4); off a boundary [16384, 1502] bf16 24 us, [16384, 1501] 38 (a lane's
// values one by one took 45 and 69), which is latency: 39% of the issue slots and 16% of
// DRAM, with 79 registers and so 24 warps an SM.
template <typename T, int kV, int kPieces>
__global__ void __launch_bounds__(32 * kWarps) k_mx8_quantize(const T* x, Rows r, uint8_t* __restrict__ codes,
                                                              uint8_t* __restrict__ scales) {
  using P = Piece<T, kV>;
  __shared__ uint4 stages[kWarps][(P::kStage * sizeof(T) + 15) / 16];
  T* stage = reinterpret_cast<T*>(stages[threadIdx.x >> 5]);
  pdl_enter();
  const int lane = threadIdx.x & 31, at = lane & 3;
  const int64_t total = r.rows * r.each, units = (total + 32 * kPieces - 1) / (32 * kPieces);
  const int64_t next = r.ld - (int64_t)r.each * 8;   // from a row's last vector to the next row's first
  const uint32_t blocks = (uint32_t)r.each / 4;
  for (int64_t u = (int64_t)blockIdx.x * kWarps + (threadIdx.x >> 5); u < units; u += (int64_t)gridDim.x * kWarps) {
    // The codes' vectors stand one after the other, whatever row they are of.
    const int64_t first = u * (32 * kPieces), t0 = divide(first, r.each), rest = total - first;
    const uint32_t v0 = (uint32_t)(first - t0 * r.each) + lane;
    const uint32_t there = rest < 32 * kPieces ? (uint32_t)rest : 32u * kPieces;
    const T* xb = x + t0 * r.ld + (int64_t)v0 * 8;
    uint8_t* cb = codes + (first + lane) * 8;
    uint8_t* sb = scales + t0 * r.scale_bytes;
    Values<T, 8> in[kPieces];
    uint32_t row[kPieces], vec[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      place<kPieces>(r, v0 + 32 * i, &row[i], &vec[i]);
      const bool live = lane + 32 * i < there;
      const int left = live ? (int)r.width - (int)vec[i] * 8 : 0;
      P::load(xb + i * 256 + row[i] * next, left, live ? row[i] : ~0u - lane, stage, lane, &in[i]);
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      float f[8];
      in[i].get(f);
      const uint32_t s = mx8_scale(mx8_block_max<8>(f));
      if (lane + 32 * i >= there) continue;
      mx8_store<8>(f, s, cb + i * 256);
      const uint32_t block = vec[i] / 4;
      uint8_t* sr = sb + row[i] * r.scale_bytes;
      if (at == 0) sr[block] = (uint8_t)s;
      if (block == blocks - 1)
        for (uint32_t b = block + 1 + at; b < r.scale_bytes; b += 4) sr[b] = 0;
    }
  }
}

// The way back, laid out the same (vectors of a row's values, no filling).
// [16384, 4096] to bf16 34 us (6.0 TB/s), [16384, 1501] 19.
template <typename T, int kV, int kPieces>
__global__ void __launch_bounds__(32 * kWarps) k_mx8_dequantize(const uint8_t* codes, const uint8_t* scales, Rows r,
                                                                T* __restrict__ x) {
  using P = Piece<T, kV>;
  __shared__ uint4 stages[kWarps][(P::kStage * sizeof(T) + 15) / 16];
  T* stage = reinterpret_cast<T*>(stages[threadIdx.x >> 5]);
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
      c[i] = *reinterpret_cast<const uint2*>(codes + t * code_bytes + (int64_t)vec[i] * 8);
      s[i] = scales[t * r.scale_bytes + vec[i] / 4];
    }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      const int64_t t = t0 + row[i];
      const bool live = t < r.rows;
      Values<T, 8> out;
      if (live) {
        const float unit = mx8_unit(s[i]);
        float f[8];
#pragma unroll
        for (int k = 0; k < 8; k += 2) {
          const float2 v = mx8_values2((k < 4 ? c[i].x : c[i].y) >> (8 * (k & 3)));
          f[k] = v.x * unit;
          f[k + 1] = v.y * unit;
        }
        out.set(f);
      }
      P::store(x + t * r.width + (int64_t)vec[i] * 8, live ? r.width - (int64_t)vec[i] * 8 : 0, live ? row[i] : ~0u - lane,
               stage, lane, out);
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

// Values of an access: eight, or two where rows are whole pairs, or one.
template <typename T>
int values_of(const void* x, int64_t ld, int64_t width) {
  const uintptr_t rows = (uintptr_t)x | (uintptr_t)(ld * (int64_t)sizeof(T));
  return row_values(rows, sizeof(T)) == 8 ? 8 : row_values(rows | (uintptr_t)(width * (int64_t)sizeof(T)), sizeof(T)) > 1 ? 2 : 1;
}

template <typename T>
cudaError_t quantize_t(const CallView& v, const T* x, int64_t ld, int64_t rows, int64_t width, uint8_t* codes,
                       uint8_t* scales, cudaStream_t st) {
  const Rows r{rows, width, ld, (int)((width + 31) / 32 * 4), (uint32_t)EBC_MX8_SCALE_BYTES(width)};
  return with_values<T>(values_of<T>(x, ld, width), [&](auto tv) {
    return with_pieces(pieces(rows * r.each, v.nsm), [&](auto tp) {
      return launch_named(v, "k_mx8_quantize", st, k_mx8_quantize<T, tv(), tp()>,
                          dim3(grid(rows * r.each, tp(), v.nsm)), dim3(32 * kWarps), 0, 1, x, r, codes, scales);
    });
  });
}

template <typename T>
cudaError_t dequantize_t(const CallView& v, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t width,
                         T* x, cudaStream_t st) {
  const Rows r{rows, width, width, (int)((width + 7) / 8), (uint32_t)EBC_MX8_SCALE_BYTES(width)};
  return with_values<T>(values_of<T>(x, width, width), [&](auto tv) {
    return with_pieces(pieces(rows * r.each, v.nsm), [&](auto tp) {
      return launch_named(v, "k_mx8_dequantize", st, k_mx8_dequantize<T, tv(), tp()>,
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
