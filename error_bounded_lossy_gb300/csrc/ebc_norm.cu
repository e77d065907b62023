// ebc_norm.cu -- the norm ahead of an expert layer: the residual's addition and
// the root-mean-square norm, to rows of the input's type and to 8-bit
// microscaled rows, and the gradients.  See include/ebc.h.
#include "ebc_mx8.cuh"

using namespace ebc;

namespace {

constexpr int kMaxThreads = 1024;
constexpr int kFewThreads = 512;   // of a row of the gradient
constexpr int kRowThreads = 256;   // of a CTA whose rows take a warp or less each

// ---- one row on a group of threads ----
// A thread has N vectors of V consecutive values: vector n * lanes + its place
// in the group.  kLanes: the lanes of a warp that a row takes; 0: whole warps
// (`lanes` threads), all of the CTA or one of several such groups.

// The group's sums of K values a thread, the same in all its threads.  `part`
// has room for two rows, so one barrier a row is enough.
// kWhole: a group is the CTA.  (Else a barrier is named by a register, for which
// a CTA is given all sixteen.)
template <int kLanes, bool kWhole, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float (*part)[K][kMaxThreads / 32], int turn, int lanes) {
#pragma unroll
  for (int off = (kLanes ? kLanes : 32) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if constexpr (kLanes == 0) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = lanes >> 5, group = kWhole ? 0 : w / warps;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) part[turn][k][w] = v[k];
    if constexpr (kWhole)
      __syncthreads();
    else
      asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(lanes) : "memory");   // (0 is __syncthreads')
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = lane < warps ? part[turn][k][group * warps + lane] : 0.f;
#pragma unroll
      for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      v[k] = s;
    }
  }
}

// ---- two fp32 numbers in one register pair, and arithmetic on both at once ----
using Two = uint64_t;
__device__ __forceinline__ Two two(float lo, float hi) {
  Two r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ __forceinline__ float2 parts_of(Two v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ Two add2(Two a, Two b) {
  Two r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two mul2(Two a, Two b) {
  Two r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ Two fma2(Two a, Two b, Two c) {
  Two r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// A thread's values are taken in chunks: one vector, or two of a single value.
template <int V>
struct Chunk {
  static constexpr int kVecs = V == 1 ? 2 : 1, kTwos = V * kVecs / 2;
};
template <typename T, int V>
__device__ __forceinline__ void widen(const Values<T, V>* v, Two (&p)[Chunk<V>::kTwos]) {
  if constexpr (V == 1) {
    p[0] = two(to_f32(v[0].e[0]), to_f32(v[1].e[0]));
  } else {
    float f[V];
    v[0].get(f);
#pragma unroll
    for (int k = 0; k < V / 2; ++k) p[k] = two(f[2 * k], f[2 * k + 1]);
  }
}
template <int V>
__device__ __forceinline__ void split(const Two (&p)[Chunk<V>::kTwos], float (&f)[V * Chunk<V>::kVecs]) {
#pragma unroll
  for (int k = 0; k < Chunk<V>::kTwos; ++k) {
    const float2 v = parts_of(p[k]);
    f[2 * k] = v.x;
    f[2 * k + 1] = v.y;
  }
}
// To the vectors' type, rounded to nearest.
template <typename T, int V>
__device__ __forceinline__ void narrow(const Two (&p)[Chunk<V>::kTwos], Values<T, V>* v) {
  float f[V * Chunk<V>::kVecs];
  split<V>(p, f);
  if constexpr (V == 1) {
    v[0].e[0] = from_f32<T>(f[0]);
    v[1].e[0] = from_f32<T>(f[1]);
  } else {
    v[0].set(f);
  }
}

// ---- rows off a vector's boundary ----
// Where all rows of a call (inputs and outputs alike) are off it by as much, they
// are still taken in whole vectors, from the boundary before a row's start on:
// kShift, with the thread's first column that much lower.  A group takes rows
// that are off by the same (every eighth row is), so it keeps its columns, and
// the weights of them.  A row's first and last vectors hold values of its
// neighbours, which are read and dropped; those of the first and last rows, which
// may have no neighbour, are read one by one.
template <int V>
__device__ __forceinline__ bool whole(int c, int width) { return c >= 0 && c + V <= width; }
template <int V>
__device__ __forceinline__ bool some(int c, int width) { return c > -V && c < width; }

// A thread's vectors of a row: which of them have columns of it, and which are
// cut by one of its ends.  (What few threads have to do is kept apart from the
// loads and stores of all, which are then issued one after the other.)
template <typename T, int V, int N, bool kShift>
struct Span {
  int c0, hop, width;   // the first vector's column, and to the next
  uint32_t in, cut;     // a bit a vector
  __device__ __forceinline__ Span(int c0, int hop, int width) : c0(c0), hop(hop), width(width), in(0), cut(0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = c0 + n * hop;
      if (kShift ? some<V>(c, width) : c < width) in |= 1u << n;
      if (kShift && some<V>(c, width) && !whole<V>(c, width)) cut |= 1u << n;
    }
  }
  __device__ __forceinline__ bool has(int n) const { return in >> n & 1; }
  // Row `p` (the thread's first column's address), or M vectors of it from vector
  // `first` on; zeros where the row is not.  Values beside the row stay until
  // clip().  edge: a row without a neighbour.
  template <int M>
  __device__ __forceinline__ void load(Values<T, V> (&v)[M], const T* p, bool live, bool edge, int first = 0) const {
    const uint32_t whole = live ? kShift && edge ? in & ~cut : in : 0u;
#pragma unroll
    for (int n = 0; n < M; ++n) {
      if (whole >> (first + n) & 1)
        v[n].load(p + (first + n) * hop);
      else
        v[n].zero();
    }
    if constexpr (kShift)
      if (live && edge && cut) ends<M>(first, [&](int n, int k) { v[n].e[k] = p[(first + n) * hop + k]; });
  }
  template <int M>
  __device__ __forceinline__ void clip(Values<T, V> (&v)[M], int first = 0) const {
    if constexpr (kShift)
      if (cut) {
#pragma unroll
        for (int n = 0; n < M; ++n) {
          const int c = c0 + (first + n) * hop;
          if (cut >> (first + n) & 1)
#pragma unroll
            for (int k = 0; k < V; ++k)
              if (c + k < 0 || c + k >= width) v[n].e[k] = from_f32<T>(0.f);
        }
      }
  }
  template <int M>
  __device__ __forceinline__ void store(const Values<T, V> (&v)[M], T* p, int first = 0) const {
#pragma unroll
    for (int n = 0; n < M; ++n)
      if ((kShift ? in & ~cut : in) >> (first + n) & 1) v[n].store(p + (first + n) * hop);
    if constexpr (kShift)
      if (cut) ends<M>(first, [&](int n, int k) { p[(first + n) * hop + k] = v[n].e[k]; });
  }
  // f(n, k) for the row's values in those of M vectors from `first` on that are cut
  template <int M, typename F>
  __device__ __forceinline__ void ends(int first, F&& f) const {
#pragma unroll
    for (int n = 0; n < M; ++n)
      if (cut >> (first + n) & 1)
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (c0 + (first + n) * hop + k >= 0 && c0 + (first + n) * hop + k < width) f(n, k);
  }
};

// A chunk's weights, of the type that the caller keeps them in; zero outside the
// row.
template <bool kShift, int V>
__device__ __forceinline__ void load_weights(const void* w, int type, int c, int hop, int width,
                                             Two (&p)[Chunk<V>::kTwos]) {
  auto get = [&](auto one) {
    using W = decltype(one);
    Values<W, V> v[Chunk<V>::kVecs];
#pragma unroll
    for (int i = 0; i < Chunk<V>::kVecs; ++i) {
      const int ci = c + i * hop;
      if constexpr (kShift) {
#pragma unroll
        for (int k = 0; k < V; ++k)
          v[i].e[k] = ci + k >= 0 && ci + k < width ? ((const W*)w)[ci + k] : from_f32<W>(0.f);
      } else {
        if (ci < width)
          v[i].load((const W*)w + ci);
        else
          v[i].zero();
      }
    }
    widen<W, V>(v, p);
  };
  if (type == EBC_F32)
    get(float());
  else if (type == EBC_BF16)
    get(__nv_bfloat16());
  else
    get(__half());
}

// A thread's weights in shared memory: its own, so there is nothing to wait for.
// Four numbers a slot, the threads' slots next to each other.
struct Slots {
  static __device__ __forceinline__ ulonglong2* at(void* base, int slot) {
    return reinterpret_cast<ulonglong2*>(base) + slot * blockDim.x + threadIdx.x;
  }
  template <int kTwos>
  static __device__ __forceinline__ void put(void* base, int q, const Two (&p)[kTwos]) {
#pragma unroll
    for (int i = 0; i < kTwos / 2; ++i) *at(base, q * (kTwos / 2) + i) = make_ulonglong2(p[2 * i], p[2 * i + 1]);
  }
  template <int kTwos>
  static __device__ __forceinline__ void get(void* base, int q, Two (&p)[kTwos]) {
#pragma unroll
    for (int i = 0; i < kTwos / 2; ++i) {
      const ulonglong2 v = *at(base, q * (kTwos / 2) + i);
      p[2 * i] = v.x;
      p[2 * i + 1] = v.y;
    }
  }
};

// How far the group's rows start past a vector's boundary (row: one of them).
template <typename T, int V, bool kShift>
__device__ __forceinline__ int shift_of(const void* rows, int64_t ld, int64_t row) {
  if constexpr (!kShift) return 0;
  return (int)(((uintptr_t)rows / sizeof(T) + (uintptr_t)(row * ld)) % V);
}

struct NormArgs {
  const void *x, *r, *w;   // r: null without a residual
  void *y, *h;             // null where not asked for
  uint8_t *codes, *scales;
  int64_t ld_x, ld_r, rows;
  int width, w_type;
  float eps;
};

// h = x + r, y = h / sqrt(mean(h^2) + eps) * w, in 32 bits: h is rounded once, to
// be kept, and y is of the sum before that rounding, rounded once to its type
// and once to 8 bits.  (A sum of squares past fp32's largest number gives a row of
// zeros, as ebc.h says.)
// Every input is read once and every output written once; bound by bandwidth:
// 8192 x 4096 bf16 with a residual 42.5 us (6.3 TB/s), 16384 rows 81 us (6.6);
// to 8 bits 41.7 and 78, both 48 and 93; off a boundary, x 4095, 53 us.  A row on
// fewer threads with more values each takes fewer joins: 16384 x 1024 25.1 us with
// eight values a thread, 22.1 with sixteen.
// An SM has 1024 threads of 16 values: left to take 68 registers the first two took
// 47.8 and 91 us.  (Single 16-bit values of more than 4096 columns spill 84 bytes in
// those 64, fp32 rows of 257 to 512 off a boundary 48.)  Wide rows: 2048 x 16384 bf16 38.4 us (on 512 threads of 32 values
// 40.6), off a boundary 2731 x 12289 41.0 (45.5).
// kAhead: without a residual there is room to load a row ahead (8192 x 4096 bf16 30.1
// -> 24.8 us, x 4095 36.2 -> 27.2, 2048 x 16384 38.3 -> 26.1; in one kernel with the
// residual's addition that loses 1 to 4%).
template <typename T, int V, int N, int kLanes, bool kShift, bool kAhead>
__global__ void __launch_bounds__(kMaxThreads) k_norm(NormArgs a) {
  __shared__ float part[2][1][kMaxThreads / 32];
  pdl_enter();
  using C = Chunk<V>;
  constexpr int kChunks = N / C::kVecs;
  const int lanes = kLanes ? kLanes : blockDim.x, at = threadIdx.x % lanes, groups = blockDim.x / lanes;
  const int64_t step = (int64_t)gridDim.x * groups;
  const int padded = (a.width + 31) / 32 * 32;
  const float share = 1.f / (float)a.width;
  // single weights stay in registers where there is room for them; vectors of them
  // are read again (a wait for them ahead of the first row: 43 -> 49 us of 8192 x 4096 bf16)
  constexpr bool kKeep = N * V <= 8 && V < 8;
  extern __shared__ ulonglong2 dynamic[];   // kShift: the weights, and what is rounded to 8 bits
  const int c0 = at * V - shift_of<T, V, kShift>(a.x, a.ld_x, blockIdx.x * groups + threadIdx.x / lanes);
  const int hop = lanes * V;   // from the thread's first column to the next
  const Span<T, V, N, kShift> span(c0, hop, a.width);
  Two kept[kKeep ? kChunks : 1][C::kTwos];
  if constexpr (kKeep)
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
      load_weights<kShift, V>(a.w, a.w_type, c0 + q * C::kVecs * hop, hop, a.width, kept[q]);
  if constexpr (kShift)
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
      Two w[C::kTwos];
      load_weights<kShift, V>(a.w, a.w_type, c0 + q * C::kVecs * hop, hop, a.width, w);
      Slots::put(dynamic, q, w);
    }
  int turn = 0;
  Values<T, V> xv[N];
  auto load_x = [&](int64_t row) {
    span.load(xv, (const T*)a.x + row * a.ld_x + c0, row < a.rows, row == 0 || row == a.rows - 1);
  };
  if constexpr (kAhead) load_x((int64_t)blockIdx.x * groups + threadIdx.x / lanes);
  // the groups of a warp, and the warps of a CTA, go through the same rounds
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + threadIdx.x / lanes;
    const bool live = row < a.rows;
    Two f[kChunks][C::kTwos];
    auto store = [&](void* rows) {
      Values<T, V> out[N];
#pragma unroll
      for (int q = 0; q < kChunks; ++q) narrow<T, V>(f[q], out + q * C::kVecs);
      if (live) span.store(out, (T*)rows + row * a.width + c0);
    };
    if constexpr (!kAhead) load_x(row);
    if (!kAhead && a.r) {
      Values<T, V> rv[N];
      span.load(rv, (const T*)a.r + row * a.ld_r + c0, live, row == 0 || row == a.rows - 1);
      span.clip(xv);
      span.clip(rv);
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        Two g[C::kTwos];
        widen<T, V>(xv + q * C::kVecs, f[q]);
        widen<T, V>(rv + q * C::kVecs, g);
#pragma unroll
        for (int k = 0; k < C::kTwos; ++k) f[q][k] = add2(f[q][k], g[k]);
      }
    } else {
      span.clip(xv);
#pragma unroll
      for (int q = 0; q < kChunks; ++q) widen<T, V>(xv + q * C::kVecs, f[q]);
      if constexpr (kAhead) load_x(row + step);
    }
    if (a.h) store(a.h);
    Two squares = 0;
#pragma unroll
    for (int q = 0; q < kChunks; ++q)
#pragma unroll
      for (int k = 0; k < C::kTwos; ++k) squares = fma2(f[q][k], f[q][k], squares);
    float sum[1] = {parts_of(squares).x + parts_of(squares).y};
    group_sum<kLanes, true>(sum, part, turn, lanes);
    const float scale = rsqrtf(sum[0] * share + a.eps);
    const Two scales2 = two(scale, scale);
#pragma unroll
    for (int q = 0; q < kChunks; ++q) {
      Two w[C::kTwos];
      if constexpr (kShift)
        Slots::get(dynamic, q, w);
      else if constexpr (!kKeep)
        load_weights<kShift, V>(a.w, a.w_type, c0 + q * C::kVecs * hop, hop, a.width, w);
#pragma unroll
      for (int k = 0; k < C::kTwos; ++k) f[q][k] = mul2(mul2(f[q][k], scales2), kKeep ? kept[kKeep ? q : 0][k] : w[k]);
    }
    if (a.y) store(a.y);
    if constexpr (kShift) {
      if (a.codes) {
        // Blocks start at column 0, vectors do not: the row goes through shared
        // memory, a word between each eight, so that neither way has lanes in the
        // same bank.
        float* y = reinterpret_cast<float*>(dynamic + kChunks * (C::kTwos / 2) * blockDim.x) +
                   (threadIdx.x / lanes) * (lanes * N * V / 8 * 9);
        if (kLanes) __syncwarp();
#pragma unroll
        for (int q = 0; q < kChunks; ++q) {
          float g[V * C::kVecs];
          split<V>(f[q], g);
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int c = c0 + q * hop + k;
            if (c >= 0) y[c + (c >> 3)] = g[k];
          }
        }
        if (kLanes)
          __syncwarp();
        else
          __syncthreads();   // (the next row's sum is between this reading and the next writing)
        uint8_t* codes = a.codes + row * padded;
        uint8_t* scales = a.scales + row * EBC_MX8_SCALE_BYTES(a.width);
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int c = (n * lanes + at) * V;
          float v[V];
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] = c + k < a.width ? y[c + (c >> 3) + k] : 0.f;
          const uint32_t s = mx8_scale(mx8_block_max<V>(v));
          if (live && c < padded) {
            mx8_store<V>(v, s, codes + c);
            if (c % 32 == 0) scales[c / 32] = (uint8_t)s;
          }
        }
      }
    } else if (a.codes) {
      uint8_t* codes = a.codes + row * padded + c0;
      uint8_t* scales = a.scales + row * EBC_MX8_SCALE_BYTES(a.width) + c0 / 32;
#pragma unroll
      for (int q = 0; q < kChunks; ++q) {
        float g[V * C::kVecs];
        split<V>(f[q], g);
        // (values past the row's end are zero, or NaN beside an infinite sum)
#pragma unroll
        for (int i = 0; i < C::kVecs; ++i) {
          const int n = q * C::kVecs + i;
          float v[V];
#pragma unroll
          for (int k = 0; k < V; ++k) v[k] = c0 + n * hop < a.width ? g[i * V + k] : 0.f;
          const uint32_t s = mx8_scale(mx8_block_max<V>(v));
          if (live && c0 + n * hop < padded) {
            mx8_store<V>(v, s, codes + n * hop);
            if (c0 % 32 == 0) scales[n * hop / 32] = (uint8_t)s;
          }
        }
      }
    }
    if (a.codes && live)
      for (int b = padded / 32 + at; b < EBC_MX8_SCALE_BYTES(a.width); b += lanes)
        a.scales[row * EBC_MX8_SCALE_BYTES(a.width) + b] = 0;
  }
}

// A weight's gradient, rounded once.
__device__ __forceinline__ void store_dweight(void* dw, int type, int64_t i, float v) {
  if (type == EBC_F32)
    ((float*)dw)[i] = v;
  else if (type == EBC_BF16)
    ((__nv_bfloat16*)dw)[i] = from_f32<__nv_bfloat16>(v);
  else
    ((__half*)dw)[i] = from_f32<__half>(v);
}

struct GradArgs {
  const void *dy, *h, *dh, *w;   // dh: null where nothing else uses h
  void *dx, *dw;
  float* parts;
  int64_t ld_dy, ld_h, ld_dh, rows;
  int width, w_type, n_parts;
  float eps;
};

// A thread's values of the rows to come, in shared memory: its own copies, which
// it alone reads, so there is nothing to wait for but its own.  One row is 16
// bytes a thread, the threads next to each other, for each 16 bytes that it has.
template <typename T, int V, int N, int kStages>
struct Ring {
  static constexpr int kParts = V * (int)sizeof(T) / 16;          // 16-byte copies of a vector
  static constexpr int kStreams = 3;                              // h, dy, dh
  static __device__ __forceinline__ uint4* at(int stage, int stream, int n, int part) {
    extern __shared__ uint4 ring[];
    return ring + (((stage * kStreams + stream) * N + n) * kParts + part) * blockDim.x + threadIdx.x;
  }
  static __device__ __forceinline__ void copy(int stage, int stream, int n, const T* src) {
#pragma unroll
    for (int i = 0; i < kParts; ++i)
      asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                       (uint32_t)__cvta_generic_to_shared(at(stage, stream, n, i))),
                   "l"(reinterpret_cast<const uint4*>(src) + i)
                   : "memory");
  }
  static __device__ __forceinline__ void get(int stage, int stream, int n, Values<T, V>* v) {
#pragma unroll
    for (int i = 0; i < kParts; ++i) {
      const uint4 r = *at(stage, stream, n, i);
      v->word[4 * i] = r.x;
      v->word[4 * i + 1] = r.y;
      v->word[4 * i + 2] = r.z;
      v->word[4 * i + 3] = r.w;
    }
  }
  static __device__ __forceinline__ T* value(int stage, int stream, int n, int k) {
    constexpr int kEach = 16 / (int)sizeof(T);
    return reinterpret_cast<T*>(at(stage, stream, n, k / kEach)) + k % kEach;
  }
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() {   // for all but the latest kStages - 1
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  }
  static __host__ __device__ size_t bytes(int threads) { return (size_t)kStages * kStreams * N * kParts * 16 * threads; }
};

// With u = h / sqrt(mean(h^2) + eps) and q = dy * w:
//   dx = (q - u * mean(q * u)) / sqrt(mean(h^2) + eps) + dh,   dw = sum over rows of dy * u.
// Both means of a row come out of one pass over it.  A thread keeps the same
// columns in every row, and with them their part of dw, so dw takes one
// partial row a CTA, which k_norm_dweight adds up in a fixed order (4 to 5 us at
// 304 CTAs; several narrow rows go to a CTA so that there are no more).
// Bound by bandwidth, if loads are in flight while a row's sums go around the
// CTA: with kStages, the rows to come are copied to shared memory meanwhile
// (without: 73 us of 8192 x 4096 bf16 with dh, so: 44, 6.1 TB/s; 16384 rows 82, 6.6).
// Not so for fp32, whose vectors are wider than such a copy (137 us with, 93
// without: 5.8 TB/s).  Weights stay in registers: read again each row, 2048 x 16384
// bf16 took 74 us, so 48 (5.6 TB/s).  Rows off a boundary: 8192 x 4095 bf16 68 us,
// 2048 x 16377 66, 8192 x 4095 fp32 103; one value an access, issue and latency (1531
// x 1001 fp32 9.4 us).  (Of 32 values a thread, single ones spill 72 to 80 bytes, rows
// off a boundary 16 to 32.)

// (Rows off a boundary take a warp more; two CTAs an SM still.)
constexpr int grad_threads(int lanes, int values, bool shift) {
  return lanes ? kRowThreads : shift && values <= 16 ? 576 : kFewThreads;
}
template <typename T, int V, int N, int kLanes, int kStages, bool kShift>
__global__ void __launch_bounds__(grad_threads(kLanes, N * V, kShift)) k_norm_grad(GradArgs a, int row_lanes) {
  using R = Ring<T, V, N, kStages>;
  using C = Chunk<V>;
  constexpr int kChunks = N / C::kVecs;
  // More values than registers hold beside dw and the weights: they are read twice, a
  // few at a time, the second time out of shared memory, or mostly of the L1 cache.
  // (Where they fit, 8192 x 4096 bf16 takes 44 us, read twice 49.)
  constexpr bool kAgain = N * V > 16 || (kShift && kStages > 0);
  constexpr int M = kAgain ? 8 / V : N;
  static_assert(!kAgain || kLanes == 0);   // (a barrier between the two)
  __shared__ float part[2][2][kMaxThreads / 32];
  pdl_enter();
  const int lanes = kLanes ? kLanes : row_lanes, at = threadIdx.x % lanes, groups = blockDim.x / lanes;
  const int64_t step = (int64_t)gridDim.x * groups;
  const float share = 1.f / (float)a.width;
  const int c0 = at * V - shift_of<T, V, kShift>(a.h, a.ld_h, blockIdx.x * groups + threadIdx.x / lanes);
  const int hop = lanes * V;   // from the thread's first column to the next
  const Span<T, V, N, kShift> span(c0, hop, a.width);
  auto request = [&](int64_t row, int stage) {   // row: of the CTA's first group
    if constexpr (kStages > 0) {
      row += threadIdx.x / lanes;
      if (row < a.rows) {
        const bool edge = row == 0 || row == a.rows - 1;
        auto copy = [&](const void* rows, int64_t ld, int stream) {
          const T* p = (const T*)rows + row * ld + c0;
#pragma unroll
          for (int n = 0; n < N; ++n)
            if ((kShift && edge ? span.in & ~span.cut : span.in) >> n & 1) R::copy(stage, stream, n, p + n * hop);
          if constexpr (kShift)
            if (edge && span.cut) span.template ends<N>(0, [&](int n, int k) { *R::value(stage, stream, n, k) = p[n * hop + k]; });
        };
        copy(a.h, a.ld_h, 0);
        copy(a.dy, a.ld_dy, 1);
        if (a.dh) copy(a.dh, a.ld_dh, 2);
      }
      R::commit();
    }
  };
  for (int i = 0; i < kStages - 1; ++i) request((int64_t)blockIdx.x * groups + i * step, i);
  // the weights stay in registers, or in shared memory where no rows to come are
  constexpr bool kSlots = kShift && kStages == 0, kKeep = !kSlots && (N * V <= 16 || V == 8);
  ulonglong2* slots = nullptr;
  if constexpr (kSlots) {
    extern __shared__ uint4 ring[];
    slots = reinterpret_cast<ulonglong2*>(ring);
  }
  Two dw[kChunks][C::kTwos], kept[kKeep ? kChunks : 1][C::kTwos];
#pragma unroll
  for (int q = 0; q < kChunks; ++q) {
#pragma unroll
    for (int k = 0; k < C::kTwos; ++k) dw[q][k] = 0;
    if constexpr (kKeep) load_weights<kShift, V>(a.w, a.w_type, c0 + q * C::kVecs * hop, hop, a.width, kept[q]);
    if constexpr (kSlots) {
      Two w[C::kTwos];
      load_weights<kShift, V>(a.w, a.w_type, c0 + q * C::kVecs * hop, hop, a.width, w);
      Slots::put(slots, q, w);
    }
  }
  auto weights = [&](int q, Two (&w)[C::kTwos]) {
    if constexpr (kSlots) {
      Slots::get(slots, q, w);
    } else if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < C::kTwos; ++k) w[k] = kept[q][k];
    } else {
      load_weights<kShift, V>(a.w, a.w_type, c0 + q * C::kVecs * hop, hop, a.width, w);
    }
  };
  int turn = 0, stage = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + threadIdx.x / lanes;
    const bool live = row < a.rows;
    const bool edge = row == 0 || row == a.rows - 1;
    // M vectors of h and dy, or of dh, from vector `first` on
    Values<T, V> hv[M], gv[M], ev[M];
    auto get_hg = [&](int first) {
      if constexpr (kStages > 0) {
#pragma unroll
        for (int n = 0; n < M; ++n) {
          if (span.has(first + n)) {
            R::get(stage, 0, first + n, &hv[n]);
            R::get(stage, 1, first + n, &gv[n]);
          } else {
            hv[n].zero();
            gv[n].zero();
          }
        }
      } else {
        span.load(hv, (const T*)a.h + row * a.ld_h + c0, live, edge, first);
        span.load(gv, (const T*)a.dy + row * a.ld_dy + c0, live, edge, first);
      }
    };
    auto get_e = [&](int first) { span.load(ev, (const T*)a.dh + row * a.ld_dh + c0, live, edge, first); };
    auto clip = [&](int first) {
      span.clip(hv, first);
      span.clip(gv, first);
    };
    if constexpr (kStages > 0) {
      request(row0 + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
      R::wait();
    }
    // (past the row's end everything is zero)
    Two squares = 0, inner = 0;
#pragma unroll
    for (int first = 0; first < N; first += M) {
      get_hg(first);
      if constexpr (kStages == 0 && !kAgain)
        if (a.dh) get_e(first);
      clip(first);
#pragma unroll
      for (int i = 0; i < M / C::kVecs; ++i) {
        const int q = first / C::kVecs + i;
        Two w[C::kTwos], h[C::kTwos], g[C::kTwos];
        weights(q, w);
        widen<T, V>(hv + i * C::kVecs, h);
        widen<T, V>(gv + i * C::kVecs, g);
#pragma unroll
        for (int k = 0; k < C::kTwos; ++k) {
          squares = fma2(h[k], h[k], squares);
          inner = fma2(mul2(g[k], w[k]), h[k], inner);
        }
      }
    }
    float sum[2] = {parts_of(squares).x + parts_of(squares).y, parts_of(inner).x + parts_of(inner).y};
    group_sum<kLanes, false>(sum, part, turn, lanes);
    const float scale = rsqrtf(sum[0] * share + a.eps), mean = sum[1] * share * scale;
    if (live) {
      const Two scale2 = two(scale, scale), mean2 = two(-mean, -mean);
      T* dx = (T*)a.dx + row * a.width + c0;
#pragma unroll
      for (int first = 0; first < N; first += M) {
        if constexpr (kAgain) {
          get_hg(first);
          if constexpr (kStages == 0)
            if (a.dh) get_e(first);
          clip(first);
        }
#pragma unroll
        for (int i = 0; i < M / C::kVecs; ++i) {
          const int q = first / C::kVecs + i;
          Two w[C::kTwos], h[C::kTwos], g[C::kTwos], d[C::kTwos];
          weights(q, w);
          widen<T, V>(hv + i * C::kVecs, h);
          widen<T, V>(gv + i * C::kVecs, g);
#pragma unroll
          for (int k = 0; k < C::kTwos; ++k) {
            const Two u = mul2(h[k], scale2);
            d[k] = mul2(fma2(u, mean2, mul2(g[k], w[k])), scale2);
            dw[q][k] = fma2(g[k], u, dw[q][k]);
          }
          if (a.dh) {
            Two e[C::kTwos];
            if constexpr (kStages > 0) {
#pragma unroll
              for (int j = 0; j < C::kVecs; ++j) R::get(stage, 2, q * C::kVecs + j, &ev[i * C::kVecs + j]);   // (stored where it is of the row)
            }
            widen<T, V>(ev + i * C::kVecs, e);
#pragma unroll
            for (int k = 0; k < C::kTwos; ++k) d[k] = add2(d[k], e[k]);
          }
          narrow<T, V>(d, gv + i * C::kVecs);
        }
        span.store(gv, dx, first);
      }
    }
    if (++stage >= kStages) stage = 0;
  }
  float sums[N * V];   // vector n's values from n * V on
#pragma unroll
  for (int q = 0; q < kChunks; ++q)
#pragma unroll
    for (int k = 0; k < C::kTwos; ++k) {
      const float2 v = parts_of(dw[q][k]);
      sums[2 * (q * C::kTwos + k)] = v.x;
      sums[2 * (q * C::kTwos + k) + 1] = v.y;
    }
  float* mine = a.parts + (int64_t)blockIdx.x * a.width;
  if (groups == 1) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = c0 + n * hop;
      if (c >= a.width) continue;
      if (gridDim.x == 1) {   // nothing to add up
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (!kShift || (c + k >= 0 && c + k < a.width)) store_dweight(a.dw, a.w_type, c + k, sums[n * V + k]);
        continue;
      }
      Values<float, V> out;
#pragma unroll
      for (int k = 0; k < V; ++k) out.e[k] = sums[n * V + k];
      if constexpr (kShift) {   // (the scratch's rows are off by another distance)
#pragma unroll
        for (int k = 0; k < V; ++k)
          if (c + k >= 0 && c + k < a.width) mine[c + k] = out.e[k];
      } else {
        out.store(mine + c);
      }
    }
  } else {
    // the CTA's groups one after the other, so that the order is the same in every run
    extern __shared__ uint4 ring[];   // (rows to come: none any more)
    float* all = reinterpret_cast<float*>(ring);
    __syncthreads();
    for (int g = 0; g < groups; ++g) {
      if ((int)threadIdx.x / lanes == g)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            const int c = c0 + n * hop + k;
            if (c >= 0 && c < a.width) all[c] = g ? all[c] + sums[n * V + k] : sums[n * V + k];
          }
      __syncthreads();
    }
    for (int c = threadIdx.x; c < a.width; c += blockDim.x)
      if (gridDim.x == 1)
        store_dweight(a.dw, a.w_type, c, all[c]);
      else
        mine[c] = all[c];
  }
}

// dw from the CTAs' partial rows: 32 columns a CTA, a warp every 32nd row.
__global__ void __launch_bounds__(1024) k_norm_dweight(const float* parts, int n_parts, int width, int type, void* dw) {
  __shared__ float sums[32][33];
  pdl_enter();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float s = 0.f;
  if (c < width)
    for (int p = w; p < n_parts; p += 32) s += parts[(int64_t)p * width + c];
  sums[w][lane] = s;
  __syncthreads();
  s = sums[lane][w];
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
  const int mine = blockIdx.x * 32 + w;
  if (lane == 0 && mine < width) store_dweight(dw, type, mine, s);
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

// A row's layout: values of a vector, vectors of a thread, lanes of a row (0:
// whole warps), and whether rows start off a vector's boundary.
template <typename T_, int V_, int N_, int kLanes_, bool kShift_>
struct Layout {
  using T = T_;
  static constexpr int V = V_, N = N_, kLanes = kLanes_;
  static constexpr bool kShift = kShift_;
};

// Calls f with the layout and the CTA's threads: a row on as few lanes as hold
// it with one vector each, then on more vectors a lane, then on whole warps.
template <typename T, typename F, int V, int N, bool kShift>
cudaError_t on_warps(int width, F&& f, Layout<T, V, N, 0, kShift> layout) {
  return f(layout, ((width + V * N - 1) / (V * N) + 31) / 32 * 32);
}
// kMost: the threads of a row with 16 values each; past them (a gradient's rows) it
// takes 32 values on half of that.
template <typename T, bool kShift, int kMost, typename F>
cudaError_t on_wide(int width, F&& f) {   // more than 512 columns
  if constexpr (16 * kMost < EBC_MAX_NORM_WIDTH)
    if (width > 16 * kMost) return on_warps<T>(width, f, Layout<T, 8, 4, 0, kShift>{});
  return on_warps<T>(width, f, Layout<T, 8, 2, 0, kShift>{});
}
template <typename T, bool kShift, int kMost, typename F>
cudaError_t with_vectors(int width, F&& f) {
  if (width <= 64) return f(Layout<T, 8, 1, 8, kShift>{}, kRowThreads);
  if (width <= 128) return f(Layout<T, 8, 1, 16, kShift>{}, kRowThreads);
  if (width <= 256) return f(Layout<T, 8, 1, 32, kShift>{}, kRowThreads);
  if (width <= 512) return f(Layout<T, 8, 2, 32, kShift>{}, kRowThreads);
  return on_wide<T, kShift, kMost>(width, f);
}
template <typename T, int kMost, typename F>
cudaError_t with_layout(int v, int width, F&& f) {
  constexpr int kValues = EBC_MAX_NORM_WIDTH / kMost;   // of a thread, in the widest rows
  if (v == 8) return with_vectors<T, false, kMost>(width, f);
  if (v == 2) {
    if (width <= 512) return f(Layout<T, 2, 8, 32, false>{}, kRowThreads);
    if (width <= 4096) return on_warps<T>(width, f, Layout<T, 2, 4, 0, false>{});
    return on_warps<T>(width, f, Layout<T, 2, kValues / 2, 0, false>{});
  }
  if (width <= 256) return f(Layout<T, 1, 8, 32, false>{}, kRowThreads);
  if (width <= 4096) return on_warps<T>(width, f, Layout<T, 1, 8, 0, false>{});
  return on_warps<T>(width, f, Layout<T, 1, kValues, 0, false>{});
}

template <typename F>
cudaError_t with_type_of(int type, F&& f) {
  if (type == EBC_F32) return f(float());
  if (type == EBC_BF16) return f(__nv_bfloat16());
  return f(__half());
}

bool shape_ok(int type, int w_type, int64_t rows, int64_t width, float eps) {
  return type_bytes(type) && type_bytes(w_type) && rows >= 0 && rows <= INT32_MAX && width >= 1 &&
         width <= EBC_MAX_NORM_WIDTH && eps >= 0.f && eps <= 3.0e38f;
}
bool ld_ok(int64_t ld, int64_t width) { return ld >= width && ld <= ((int64_t)1 << 40); }

// What one access takes: 8 values where all rows and the weight allow it, else 2
// or 1; and whether all rows are off a vector's boundary by as much.
struct Places {
  uintptr_t all = 0, first = 0, stride = 0;
  bool alike = true, any = false;
  int elem;
  // (a row's last vector must not reach into what is beside it)
  Places(int elem, int64_t width) : all((uintptr_t)(width * elem)), elem(elem) {}
  void add(const void* p, int64_t ld) {
    if (!p) return;
    const uintptr_t a = (uintptr_t)p, s = (uintptr_t)(ld * elem), unit = (uintptr_t)(8 * elem);
    if (any && ((a - first) % unit || (s - stride) % unit)) alike = false;
    if (!any) {
      first = a;
      stride = s;
    }
    any = true;
    all |= a | s;
  }
  int values(const void* w, int w_elem) const {
    const int a = row_values(all, elem), b = row_values((uintptr_t)w, w_elem);
    return a < b ? a : b;
  }
  // Whether such rows can be taken in whole vectors all the same (with up to 7
  // columns more, and a row's neighbours no nearer than a vector).  Not so are rows
  // of a padded buffer, whose outputs are dense and off by another distance: 8192 x
  // 4095 bf16 of rows of 4096 take 173 us with a residual, of rows of 4095 53.
  bool shifts(int64_t width) const { return alike && width >= 8 && width + 7 <= EBC_MAX_NORM_WIDTH; }
};

}  // namespace

extern "C" {

int ebc_norm(ebc_ctx* ctx, const void* d_x, int64_t ld_x, const void* d_residual, int64_t ld_residual, int type,
             const void* d_weight, int weight_type, int64_t rows, int64_t width, float eps, void* d_y, void* d_h,
             uint8_t* d_codes, uint8_t* d_scales, void* stream) {
  if (!ctx || !shape_ok(type, weight_type, rows, width, eps) || !ld_ok(ld_x, width) ||
      (d_residual && !ld_ok(ld_residual, width)) || (!d_codes != !d_scales))
    return EBC_ERR_INVALID_ARG;
  const int b = type_bytes(type), wb = type_bytes(weight_type);
  if (rows > 0 && (!d_x || !aligned(d_x, b) || !aligned(d_residual, b) || !d_weight || !aligned(d_weight, wb) ||
                   !aligned(d_y, b) || !aligned(d_h, b) || !aligned(d_codes, 16) || !aligned(d_scales, 16) ||
                   (!d_y && !d_codes)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || rows == 0) return rc;
  const NormArgs a{d_x, d_residual, d_weight, d_y, d_h, d_codes, d_scales, ld_x, ld_residual, rows,
                   (int)width, weight_type, eps};
  Places at(b, width);
  at.add(d_x, ld_x);
  at.add(d_residual, ld_residual);
  at.add(d_y, width);
  at.add(d_h, width);
  return cuda_code(with_type_of(type, [&](auto one) {
    using T = decltype(one);
    auto run = [&](auto l, int threads, auto kernel, bool ahead) {
      using L = decltype(l);
      const int groups = L::kLanes ? threads / L::kLanes : 1;
      // (a multiple of eight, so that a group's rows are all off by as much; with
      // weights kept, or a row ahead, no more than are resident)
      const int64_t want = (rows + groups - 1) / groups;
      const int64_t most = ((int64_t)v.nsm * (L::kShift || ahead ? 1024 / threads : 2048 / threads * 2)) & ~7ll;
      size_t smem = 0;
      if constexpr (L::kShift) {
        constexpr int kWeights = 4 * L::N * L::V, kRow = kWeights / 8 * 9;   // bytes a thread
        const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   (kWeights + kRow) * kMaxThreads);
        if (e != cudaSuccess) return e;
        smem = (size_t)threads * (d_codes ? kWeights + kRow : kWeights);
      }
      return launch_named(v, "k_norm", st, kernel, dim3((unsigned)(want < most || most < 8 ? want : most)),
                          dim3(threads), smem, 1, a);
    };
    auto launch = [&](auto l, int threads) {
      using L = decltype(l);
      if constexpr (L::V == 8)
        if (!d_residual) return run(l, threads, k_norm<typename L::T, L::V, L::N, L::kLanes, L::kShift, true>, true);
      return run(l, threads, k_norm<typename L::T, L::V, L::N, L::kLanes, L::kShift, false>, false);
    };
    const int vals = at.values(d_weight, wb);
    return vals < 8 && at.shifts(width) ? with_vectors<T, true, kMaxThreads>((int)width + 7, launch)
                                        : with_layout<T, kMaxThreads>(vals, (int)width, launch);
  }));
}

int ebc_norm_grad(ebc_ctx* ctx, const void* d_dy, int64_t ld_dy, const void* d_h, int64_t ld_h, const void* d_dh,
                  int64_t ld_dh, int type, const void* d_weight, int weight_type, int64_t rows, int64_t width,
                  float eps, void* d_dx, void* d_dweight, float* d_scratch, void* stream) {
  if (!ctx || !shape_ok(type, weight_type, rows, width, eps) || !ld_ok(ld_dy, width) || !ld_ok(ld_h, width) ||
      (d_dh && !ld_ok(ld_dh, width)))
    return EBC_ERR_INVALID_ARG;
  const int b = type_bytes(type), wb = type_bytes(weight_type);
  if (!d_dweight || !aligned(d_dweight, wb) ||
      (rows > 0 && (!d_dy || !aligned(d_dy, b) || !d_h || !aligned(d_h, b) || !aligned(d_dh, b) || !d_weight ||
                    !aligned(d_weight, wb) || !d_dx || !aligned(d_dx, b) || !d_scratch || !aligned(d_scratch, 16))))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc) return rc;
  GradArgs a{d_dy, d_h, d_dh, d_weight, d_dx, d_dweight, d_scratch, ld_dy, ld_h, ld_dh, rows, (int)width, weight_type,
             0, eps};
  cudaError_t e = cudaSuccess;
  if (rows > 0) {
    Places at(b, width);
    at.add(d_dy, ld_dy);
    at.add(d_h, ld_h);
    at.add(d_dh, ld_dh);
    at.add(d_dx, width);
    int vals = at.values(d_weight, wb);
    // (fp32 partial rows start where the scratch's 16 bytes allow: whole vectors of 8 want 32)
    const int vals_s = row_values((uintptr_t)d_scratch | (uintptr_t)(width * 4), 4);
    if (vals > vals_s) vals = vals_s;
    // Rows off the boundary in whole vectors where it takes less time: very wide ones,
    // and many of more than 512 values (us with dh, single values / so, bf16: 600 x
    // 1001 7.9 / 8.4, 1531 x 1001 11.0 / 11.0, 8192 x 1001 48 / 23, 256 x 4095 8.8 / 10.6,
    // 1024 x 4095 25.5 / 17.5, 64 x 8101 27.8 / 11.1, 16384 x 101 11.8 / 21.9; fp32: 2048 x
    // 1001 11.5 / 12.7, 8192 x 1001 33 / 32, 2048 x 4095 38.6 / 34.0, 64 x 8101 22.6 / 11.8).
    const bool many = rows * width >= (b == 2 ? 3 << 19 : 1 << 22);
    const bool shift = vals < 8 && at.shifts(width) && (width > 4096 || (width > 512 && many));
    e = with_type_of(type, [&](auto one) {
      using T = decltype(one);
      auto launch = [&](auto l, int threads) {
        using L = decltype(l);
        // A row a CTA of whole vectors: the rows to come in shared memory.  Three
        // stages: with two CTAs of 256 threads an SM that is 98 KB in flight (8192 x
        // 4096 bf16 with dh 45.0 us; 45.5 with two stages, 47.8 with four), and with
        // one of 448 threads 86 KB (8192 x 7168: 73.4; 80.9, 72.7).
        constexpr int kStages = L::kLanes || L::V < 8 || sizeof(typename L::T) > 2 ? 0 : L::N == 2 ? 3 : 2;
        const auto kernel = k_norm_grad<typename L::T, L::V, L::N, L::kLanes, kStages, L::kShift>;
        // Rows that take less than 256 threads: several in a CTA.
        const int lanes = L::kLanes ? L::kLanes : threads, groups = L::kLanes || threads <= 128 ? kRowThreads / lanes : 1;
        threads = groups * lanes;
        // All CTAs at once, as many on each SM as registers (16-bit vectors 63, fp32 ones
        // 68, pairs 74, single values 101), shared memory and the scratch's rows allow (in
        // two turns 1531 x 1001 fp32 with dh took 11.3 us, so 9.4; 131072 x 63 57 and 43).
        constexpr bool kHalf = sizeof(typename L::T) == 2;
        constexpr int kFit = L::N * L::V > 8 ? (L::kLanes ? kFewThreads : grad_threads(0, L::N * L::V, L::kShift))
                             : L::V == 1 && (kHalf || !L::kLanes) ? 512
                             : L::V == 8 && kHalf                 ? 1024
                                                                  : 768;
        int64_t each = kFit / threads < 1 ? 1 : kFit / threads;
        // where the groups' sums are added up
        size_t smem = groups > 1 ? (size_t)4 * L::N * L::V * lanes : 0;
        if constexpr (L::kShift && kStages == 0) {   // the weights, before that
          smem = (size_t)4 * L::N * L::V * threads;
          const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     4 * L::N * L::V * grad_threads(0, L::N * L::V, true));
          if (e != cudaSuccess) return e;
        }
        if constexpr (kStages > 0) {
          const size_t ring = Ring<typename L::T, L::V, L::N, kStages>::bytes(threads);
          constexpr int kMost = 226 * 1024;   // of an SM's 228 KB (each CTA has 1 KB of its own)
          if (ring > smem) smem = ring;
          if (each * (int64_t)(smem + 2048) > kMost) each = kMost / (int64_t)(smem + 2048);
          // so much that no SM takes more: the kernel before may still fill some of them
          smem = (size_t)(kMost / each - 2048) & ~(size_t)127;
          const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kMost - 2048);
          if (e != cudaSuccess) return e;
        }
        const int64_t want = (rows + groups - 1) / groups;
        int64_t most = (int64_t)v.nsm * each;
        if (most > EBC_NORM_GRAD_PARTS) most = EBC_NORM_GRAD_PARTS;
        most = most < 8 ? 1 : most & ~7ll;   // (so that a group's rows are all off by as much)
        a.n_parts = (int)(want < most ? want : most);
        return launch_named(v, "k_norm_grad", st, kernel, dim3((unsigned)a.n_parts), dim3(threads), smem, 1, a, lanes);
      };
      if (shift) return on_wide<T, true, kFewThreads>((int)width + 7, launch);
      return with_layout<T, kFewThreads>(vals, (int)width, launch);
    });
  }
  if (e == cudaSuccess && a.n_parts != 1)
    e = launch_named(v, "k_norm_dweight", st, k_norm_dweight, dim3((unsigned)((width + 31) / 32)), dim3(1024), 0, 1,
                     d_scratch, a.n_parts, (int)width, weight_type, d_dweight);
  return cuda_code(e);
}

}  // extern "C"
