// ebc_mx4.cu -- rows to 4-bit microscaled values and back, alone and on the
// way into the experts' sending buffer.  See include/ebc.h for the format.
#include "ebc_mx4.cuh"

using namespace ebc;

namespace {

constexpr int kMxWarps = 8;
constexpr int kLane = 8;            // consecutive values of a lane; a block is four lanes
constexpr int kPiece = 32 * kLane;  // consecutive values of a warp

// a / b; most often in 32 bits, a fifth of the instructions
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return a <= UINT32_MAX ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}

// Chunks of a row, its scales' filling included.
__host__ __device__ __forceinline__ int64_t scale_chunks(int64_t width, int chunk) {
  return (EBC_MX4_SCALE_BYTES(width) * 32 + chunk - 1) / chunk;
}

// Eight values of a row as they are in memory.
template <typename T>
struct Eight {
  static constexpr int kWords = kLane * (int)sizeof(T) / 4;
  union {
    uint32_t word[kWords];
    T e[kLane];
  };
  __device__ __forceinline__ Eight() {}
};
// A warp's piece between memory and its lanes' eights; `left`: the row's values
// from the lane's first on (values past the row's end are zero, or not written).
// kV = 8 * sizeof(T): rows whose eights are aligned, one load or store a lane.
// Other rows go through the warp's own piece of shared memory in vectors of kV
// bytes, the lanes next to each other: a lane that took its eight values one by
// one touched 16 sectors an access ([8192, 1501] bf16: 49 us to quantize and
// read back).
template <typename T, int kV>
struct Piece {
  static constexpr bool kDirect = kV == kLane * (int)sizeof(T);
  using Raw_ = typename Raw<kDirect ? 16 : kV>::T;

  // row: the piece's first value; left0: the row's values from there on
  static __device__ __forceinline__ void load(const T* row, int64_t left0, int lane, T* stage, Eight<T>* v) {
    if constexpr (kDirect) {
      const T* p = row + lane * kLane;
      const int64_t left = left0 - lane * kLane;
      if (left >= kLane) {
        if constexpr (sizeof(T) == 4)
          asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                       : "=r"(v->word[0]), "=r"(v->word[1]), "=r"(v->word[2]), "=r"(v->word[3]), "=r"(v->word[4]),
                         "=r"(v->word[5]), "=r"(v->word[6]), "=r"(v->word[7])
                       : "l"(p));
        else
          asm volatile("ld.global.v4.b32 {%0, %1, %2, %3}, [%4];"
                       : "=r"(v->word[0]), "=r"(v->word[1]), "=r"(v->word[2]), "=r"(v->word[3])
                       : "l"(p));
      } else {
#pragma unroll
        for (int k = 0; k < kLane; ++k) v->e[k] = k < left ? p[k] : from_f32<T>(0.f);
      }
    } else {
      constexpr int kN = kV / (int)sizeof(T), kSteps = kLane / kN;
      Raw_ r[kSteps];
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int at = (i * 32 + lane) * kN;
        r[i] = at < left0 ? *reinterpret_cast<const Raw_*>(row + at) : Raw_{};
      }
      __syncwarp();   // the last piece has been taken
#pragma unroll
      for (int i = 0; i < kSteps; ++i) *reinterpret_cast<Raw_*>(stage + (i * 32 + lane) * kN) = r[i];
      __syncwarp();
#pragma unroll
      for (int k = 0; k < Eight<T>::kWords; ++k) v->word[k] = reinterpret_cast<const uint32_t*>(stage + lane * kLane)[k];
    }
  }
  static __device__ __forceinline__ void store(T* row, int64_t left0, int lane, T* stage, const Eight<T>& v) {
    if constexpr (kDirect) {
      T* p = row + lane * kLane;
      const int64_t left = left0 - lane * kLane;
      if (left >= kLane) {
        if constexpr (sizeof(T) == 4)
          asm volatile("st.global.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(v.word[0]), "r"(v.word[1]),
                       "r"(v.word[2]), "r"(v.word[3]), "r"(v.word[4]), "r"(v.word[5]), "r"(v.word[6]), "r"(v.word[7]),
                       "l"(p)
                       : "memory");
        else
          asm volatile("st.global.v4.b32 [%4], {%0, %1, %2, %3};" ::"r"(v.word[0]), "r"(v.word[1]), "r"(v.word[2]),
                       "r"(v.word[3]), "l"(p)
                       : "memory");
      } else {
#pragma unroll
        for (int k = 0; k < kLane; ++k)
          if (k < left) p[k] = v.e[k];
      }
    } else {
      constexpr int kN = kV / (int)sizeof(T), kSteps = kLane / kN;
      __syncwarp();
#pragma unroll
      for (int k = 0; k < Eight<T>::kWords; ++k) reinterpret_cast<uint32_t*>(stage + lane * kLane)[k] = v.word[k];
      __syncwarp();
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const int at = (i * 32 + lane) * kN;
        if (at < left0) *reinterpret_cast<Raw_*>(row + at) = *reinterpret_cast<const Raw_*>(stage + at);
      }
    }
  }
};

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
  const float inv = mx4_inverse(s);
  float u[kLane];
#pragma unroll
  for (int k = 0; k < kLane; ++k) u[k] = to_f32(v.e[k]) * inv;
  return s == 255u ? 0u : mx4_codes(u);
}

// A warp takes kPieces runs of 256 consecutive values of a row, eight a lane,
// all of them in flight at once.  With kRoute each token's codes go to the
// rows of its choices: quantized once, written `top` times, and rows past the
// last expert's are zero.
// 16 or 32 bits are read and 4.25 written a value: bound by bandwidth, for 16-bit
// types by issue as much (71% of the cycles issue, 60% of DRAM's rate).  [16384, 4096] bf16: 29 us (5.9 TB/s);
// [8192, 3328] fp32: 22 us (5.6 TB/s).
template <typename T, int kV, bool kRoute, int kPieces>
__global__ void __launch_bounds__(32 * kMxWarps) k_mx4_quantize(const T* x, int64_t ld, int64_t rows,
                                                                int64_t width, int top,
                                                                const int32_t* place,
                                                                const int32_t* offsets, int E,
                                                                uint8_t* __restrict__ codes,
                                                                uint8_t* __restrict__ scales, Glob* glob) {
  using P = Piece<T, kV>;
  __shared__ uint4 s_stage[P::kDirect ? 1 : kMxWarps * kPiece * sizeof(T) / 16];
  T* stage = reinterpret_cast<T*>(s_stage) + (P::kDirect ? 0 : (threadIdx.x >> 5) * kPiece);
  pdl_enter();
  constexpr int kChunk = kPieces * kPiece;
  const int lane = threadIdx.x & 31, quad = lane >> 2, j4 = lane & 3;
  const int64_t code_bytes = EBC_MX4_CODE_BYTES(width), scale_bytes = EBC_MX4_SCALE_BYTES(width);
  const int64_t chunks = scale_chunks(width, kChunk);
  const int64_t n = rows * top;
  int64_t live = n;
  if (kRoute) {
    live = offsets[E];
    live = live < 0 ? 0 : live < n ? live : n;
  }
  const int64_t units = (rows + (n - live)) * chunks;
  for (int64_t u = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kMxWarps) {
    const int64_t t = divide(u, chunks), h0 = (u - t * chunks) * kChunk, left = width - h0 - lane * kLane;
    uint32_t c[kPieces], s[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i) c[i] = s[i] = 0u;
    if (!kRoute || t < rows) {
      const T* src = x + t * ld + h0;
      Eight<T> v[kPieces];
#pragma unroll
      for (int i = 0; i < kPieces; ++i) P::load(src + i * kPiece, width - h0 - i * kPiece, lane, stage, &v[i]);
#pragma unroll
      for (int i = 0; i < kPieces; ++i) {
        c[i] = encode8(v[i], &s[i]);
        // a block past the row's end; a block's lanes agree on that
        if (left + j4 * kLane - i * kPiece <= 0) s[i] = 0u;
      }
    }
    // of four pieces' scale bytes a block's lanes store one each
    uint32_t mine[(kPieces + 3) / 4];
#pragma unroll
    for (int q = 0; q < (kPieces + 3) / 4; ++q) {
      uint32_t all = 0;
#pragma unroll
      for (int i = 0; i < 4 && 4 * q + i < kPieces; ++i) all |= s[4 * q + i] << (8 * i);
      mine[q] = all >> (8 * j4);
    }
    const int64_t code_left = code_bytes - h0 / 2 - lane * 4, scale_left = scale_bytes - h0 / 32 - j4 * 8 - quad;
    auto store = [&](int64_t r) {
      uint8_t* cr = codes + r * code_bytes + h0 / 2 + lane * 4;
      uint8_t* sr = scales + r * scale_bytes + h0 / 32 + j4 * 8 + quad;
#pragma unroll
      for (int i = 0; i < kPieces; ++i)
        if (i * (kPiece / 2) < code_left) *reinterpret_cast<uint32_t*>(cr + i * (kPiece / 2)) = c[i];
#pragma unroll
      for (int q = 0; q < (kPieces + 3) / 4; ++q)
        if (4 * q + j4 < kPieces && q * 32 < scale_left) sr[q * 32] = (uint8_t)mine[q];
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

// The way back: eight codes a lane, kPieces runs of 256 values a warp.  Bound
// by the bandwidth of the writes ([8192, 3328] to fp32: 20 us, 6.1 TB/s), to
// 16-bit types by issue (71% of the cycles, DRAM at 49%).
template <typename T, int kV, int kPieces>
__global__ void __launch_bounds__(32 * kMxWarps) k_mx4_dequantize(const uint8_t* codes,
                                                                  const uint8_t* scales, int64_t rows,
                                                                  int64_t width, T* __restrict__ x) {
  using P = Piece<T, kV>;
  __shared__ uint4 s_stage[P::kDirect ? 1 : kMxWarps * kPiece * sizeof(T) / 16];
  T* stage = reinterpret_cast<T*>(s_stage) + (P::kDirect ? 0 : (threadIdx.x >> 5) * kPiece);
  pdl_enter();
  constexpr int kChunk = kPieces * kPiece;
  const int lane = threadIdx.x & 31;
  const int64_t chunks = (width + kChunk - 1) / kChunk;
  const int64_t code_bytes = EBC_MX4_CODE_BYTES(width), scale_bytes = EBC_MX4_SCALE_BYTES(width);
  for (int64_t u = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5); u < rows * chunks;
       u += (int64_t)gridDim.x * kMxWarps) {
    const int64_t t = divide(u, chunks), h0 = (u - t * chunks) * kChunk, left = width - h0 - lane * kLane;
    const uint8_t* cr = codes + t * code_bytes + h0 / 2 + lane * 4;
    const uint8_t* sr = scales + t * scale_bytes + h0 / 32 + (lane >> 2);
    T* dst = x + t * width + h0;
    uint32_t c[kPieces], s[kPieces];
#pragma unroll
    for (int i = 0; i < kPieces; ++i)
      if (i * kPiece < left) {
        c[i] = *reinterpret_cast<const uint32_t*>(cr + i * (kPiece / 2));
        s[i] = sr[i * (kPiece / 32)];
      }
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
      if (i * kPiece >= width - h0) break;
      Eight<T> o;
      if (i * kPiece < left) {
        const float unit = mx4_unit(s[i]);
        __half2 h[4];
        mx4_values(c[i], h);
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const float2 f = __half22float2(h[k]);
          o.e[2 * k] = from_f32<T>(f.x * unit);
          o.e[2 * k + 1] = from_f32<T>(f.y * unit);
        }
      }
      P::store(dst + i * kPiece, width - h0 - i * kPiece, lane, stage, o);
    }
  }
}

// Rows of at most 128 values, which would leave most lanes of a piece idle:
// 4, 8 or 16 lanes a row (1 << lanes_log2), kNarrow runs of rows a warp.  In
// pieces, 16384 bf16 rows of 64 or of 128 took 18.9 us to quantize and 5.4 to
// read back; so they take less than 4.9 and 3.8, the call's time on the host.
constexpr int kNarrowWidth = 128, kNarrow = 4;

// A lane's eight values of a short row, in 16-byte loads where `wide`.
template <typename T>
__device__ __forceinline__ void load_narrow(const T* p, int64_t left, bool wide, Eight<T>* v) {
  if (wide && left >= kLane) {
#pragma unroll
    for (int i = 0; i < Eight<T>::kWords / 4; ++i) {
      const uint4 r = reinterpret_cast<const uint4*>(p)[i];
      v->word[4 * i] = r.x;
      v->word[4 * i + 1] = r.y;
      v->word[4 * i + 2] = r.z;
      v->word[4 * i + 3] = r.w;
    }
  } else {
#pragma unroll
    for (int k = 0; k < kLane; ++k) v->e[k] = k < left ? p[k] : from_f32<T>(0.f);
  }
}

template <typename T, bool kRoute>
__global__ void __launch_bounds__(32 * kMxWarps) k_mx4_quantize_narrow(const T* x, int64_t ld,
                                                                       int64_t rows, int width, int lanes_log2,
                                                                       bool wide, int top,
                                                                       const int32_t* place,
                                                                       const int32_t* offsets, int E,
                                                                       uint8_t* __restrict__ codes,
                                                                       uint8_t* __restrict__ scales, Glob* glob) {
  pdl_enter();
  const int lane = threadIdx.x & 31, lanes = 1 << lanes_log2, at = lane & (lanes - 1), each = 32 >> lanes_log2;
  const int code_bytes = EBC_MX4_CODE_BYTES(width);
  const int64_t n = rows * top;
  int64_t live = n;
  if (kRoute) {
    live = offsets[E];
    live = live < 0 ? 0 : live < n ? live : n;
  }
  const int64_t total = rows + (n - live), units = (total + each * kNarrow - 1) / (each * kNarrow);
  for (int64_t u = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kMxWarps) {
    Eight<T> v[kNarrow];
#pragma unroll
    for (int i = 0; i < kNarrow; ++i) {
      const int64_t t = (u * kNarrow + i) * each + (lane >> lanes_log2);
      load_narrow(x + t * ld + at * kLane, t < rows ? width - at * kLane : 0, wide, &v[i]);
    }
#pragma unroll
    for (int i = 0; i < kNarrow; ++i) {
      const int64_t t = (u * kNarrow + i) * each + (lane >> lanes_log2);
      uint32_t s;
      const uint32_t c = encode8(v[i], &s);
      if (t >= rows || (at & ~3) * kLane >= width) s = 0u;
      uint32_t word = 0;   // the row's scale bytes
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t b = __shfl_sync(0xffffffffu, s, (lane - at + 4 * k) & 31);
        if (4 * k < lanes) word |= b << (8 * k);
      }
      auto store = [&](int64_t r) {
        if (at * 4 < code_bytes) *reinterpret_cast<uint32_t*>(codes + r * code_bytes + at * 4) = c;
        if (at == 0) *reinterpret_cast<uint4*>(scales + r * 16) = make_uint4(word, 0u, 0u, 0u);
      };
      if (t >= total) continue;
      if (!kRoute) {
        store(t);
      } else if (t < rows) {
        for (int j = 0; j < top; ++j) {
          const int32_t p = place[t * top + j];
          if (p >= n && at == 0) record_error(glob, EBC_ERR_INVALID_ARG);
          if (p >= 0 && p < n) store(p);
        }
      } else {
        store(live + (t - rows));
      }
    }
  }
}

template <typename T>
__global__ void __launch_bounds__(32 * kMxWarps) k_mx4_dequantize_narrow(const uint8_t* codes,
                                                                         const uint8_t* scales,
                                                                         int64_t rows, int width, int lanes_log2,
                                                                         bool wide, T* __restrict__ x) {
  pdl_enter();
  const int lane = threadIdx.x & 31, lanes = 1 << lanes_log2, at = lane & (lanes - 1), each = 32 >> lanes_log2;
  const int code_bytes = EBC_MX4_CODE_BYTES(width), left = width - at * kLane;
  const int64_t units = (rows + each * kNarrow - 1) / (each * kNarrow);
  for (int64_t u = (int64_t)blockIdx.x * kMxWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kMxWarps) {
    uint32_t c[kNarrow], s[kNarrow];
#pragma unroll
    for (int i = 0; i < kNarrow; ++i) {
      const int64_t t = (u * kNarrow + i) * each + (lane >> lanes_log2);
      if (t < rows && left > 0) {
        c[i] = *reinterpret_cast<const uint32_t*>(codes + t * code_bytes + at * 4);
        s[i] = scales[t * 16 + (at >> 2)];
      }
    }
#pragma unroll
    for (int i = 0; i < kNarrow; ++i) {
      const int64_t t = (u * kNarrow + i) * each + (lane >> lanes_log2);
      if (t >= rows || left <= 0) continue;
      const float unit = mx4_unit(s[i]);
      __half2 h[4];
      mx4_values(c[i], h);
      Eight<T> o;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float2 f = __half22float2(h[k]);
        o.e[2 * k] = from_f32<T>(f.x * unit);
        o.e[2 * k + 1] = from_f32<T>(f.y * unit);
      }
      T* dst = x + t * width + at * kLane;
      if (wide && left >= kLane) {
#pragma unroll
        for (int q = 0; q < Eight<T>::kWords / 4; ++q)
          reinterpret_cast<uint4*>(dst)[q] =
              make_uint4(o.word[4 * q], o.word[4 * q + 1], o.word[4 * q + 2], o.word[4 * q + 3]);
      } else {
#pragma unroll
        for (int k = 0; k < kLane; ++k)
          if (k < left) dst[k] = o.e[k];
      }
    }
  }
}

// Lanes of a short row: its blocks', four each.
int narrow_lanes_log2(int64_t width) { return width <= 32 ? 2 : width <= 64 ? 3 : 4; }

// Pieces of a warp: as many (up to `most`) as leave 24 warps for each SM.  A
// warp's own cost (about 150 instructions) is spread over them, and their
// loads overlap: [16384, 4096] bf16 takes 52 us with one, 40 with two, 32 with
// four and 29 with eight; [1531, 1056] fp16 3.8 with one, 3.5 with two, 4.4
// with four.
int pieces(int64_t rows, int64_t width, int nsm, int most) {
  int p = most;
  while (p > 1 && rows * scale_chunks(width, p * kPiece) < (int64_t)nsm * 24) p /= 2;
  return p;
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// CTAs for `units` warps of work, at most two full turns of the machine; the
// kernels loop beyond that.
unsigned mx_grid(int64_t units, int nsm) {
  const int64_t want = (units + kMxWarps - 1) / kMxWarps, most = (int64_t)nsm * 8 * 2;
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

bool mx_rows_ok(int64_t rows, int64_t width) {
  return rows >= 0 && rows <= INT32_MAX && width >= 1 && width <= (1 << 24);
}

template <typename T, int kV, bool kRoute, int kPieces>
cudaError_t quantize_launch(const CallView& v, const void* x, int64_t ld, int64_t rows, int64_t width, int top,
                            const int32_t* place, const int32_t* offsets, int E, uint8_t* codes, uint8_t* scales,
                            cudaStream_t st) {
  return launch_named(v, kRoute ? "k_mx4_dispatch" : "k_mx4_quantize", st,
                      k_mx4_quantize<T, kV, kRoute, kPieces>,
                      dim3(mx_grid(rows * scale_chunks(width, kPieces * kPiece), v.nsm)), dim3(32 * kMxWarps), 0, 1,
                      (const T*)x, ld, rows, width, top, place, offsets, E, codes, scales, v.glob);
}

template <typename T, bool kRoute>
cudaError_t quantize_t(const CallView& v, const void* x, int64_t ld, int64_t rows, int64_t width, int top,
                       const int32_t* place, const int32_t* offsets, int E, uint8_t* codes, uint8_t* scales,
                       cudaStream_t st) {
  constexpr int kMost = sizeof(T) == 2 ? 8 : 4, kV = kLane * (int)sizeof(T);
  const uintptr_t rows_at = (uintptr_t)x | (uintptr_t)(ld * (int64_t)sizeof(T));
  if (width <= kNarrowWidth) {
    const int lanes = narrow_lanes_log2(width);
    const int64_t units = (rows + (32 >> lanes) * kNarrow - 1) / ((32 >> lanes) * kNarrow);
    return launch_named(v, kRoute ? "k_mx4_dispatch" : "k_mx4_quantize", st, k_mx4_quantize_narrow<T, kRoute>,
                        dim3(mx_grid(units, v.nsm)), dim3(32 * kMxWarps), 0, 1, (const T*)x, ld, rows, (int)width,
                        lanes, rows_at % 16 == 0, top, place, offsets, E, codes, scales, v.glob);
  }
  if (rows_at % kV != 0) {
    // vectors of two 16-bit values where a row is whole vectors, else single values
    if (sizeof(T) == 2 && (rows_at | (uintptr_t)(width * (int64_t)sizeof(T))) % 4 == 0)
      return quantize_launch<T, 4, kRoute, 2>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
    return quantize_launch<T, (int)sizeof(T), kRoute, 2>(v, x, ld, rows, width, top, place, offsets, E, codes, scales,
                                                         st);
  }
  switch (pieces(rows, width, v.nsm, kMost)) {
    case 1: return quantize_launch<T, kV, kRoute, 1>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
    case 2: return quantize_launch<T, kV, kRoute, 2>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
    case 4: return quantize_launch<T, kV, kRoute, 4>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
    default:
      return quantize_launch<T, kV, kRoute, kMost>(v, x, ld, rows, width, top, place, offsets, E, codes, scales, st);
  }
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

template <typename T, int kV, int kPieces>
cudaError_t dequantize_launch(const CallView& v, const uint8_t* codes, const uint8_t* scales, int64_t rows,
                              int64_t width, void* x, cudaStream_t st) {
  const int64_t chunk = kPieces * kPiece;
  return launch_named(v, "k_mx4_dequantize", st, k_mx4_dequantize<T, kV, kPieces>,
                      dim3(mx_grid(rows * ((width + chunk - 1) / chunk), v.nsm)), dim3(32 * kMxWarps), 0, 1, codes,
                      scales, rows, width, (T*)x);
}

template <typename T>
cudaError_t dequantize_t(const CallView& v, const uint8_t* codes, const uint8_t* scales, int64_t rows, int64_t width,
                         void* x, cudaStream_t st) {
  constexpr int kV = kLane * (int)sizeof(T);
  const uintptr_t rows_at = (uintptr_t)x | (uintptr_t)(width * (int64_t)sizeof(T));
  if (width <= kNarrowWidth) {
    const int lanes = narrow_lanes_log2(width);
    const int64_t units = (rows + (32 >> lanes) * kNarrow - 1) / ((32 >> lanes) * kNarrow);
    return launch_named(v, "k_mx4_dequantize", st, k_mx4_dequantize_narrow<T>, dim3(mx_grid(units, v.nsm)),
                        dim3(32 * kMxWarps), 0, 1, codes, scales, rows, (int)width, lanes, rows_at % 16 == 0, (T*)x);
  }
  if (rows_at % kV != 0) {
    if (sizeof(T) == 2 && rows_at % 4 == 0) return dequantize_launch<T, 4, 2>(v, codes, scales, rows, width, x, st);
    return dequantize_launch<T, (int)sizeof(T), 2>(v, codes, scales, rows, width, x, st);
  }
  switch (pieces(rows, width, v.nsm, 4)) {
    case 1: return dequantize_launch<T, kV, 1>(v, codes, scales, rows, width, x, st);
    case 2: return dequantize_launch<T, kV, 2>(v, codes, scales, rows, width, x, st);
    default: return dequantize_launch<T, kV, 4>(v, codes, scales, rows, width, x, st);
  }
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
