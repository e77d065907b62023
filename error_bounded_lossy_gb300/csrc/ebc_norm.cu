// ebc_norm.cu -- the norm ahead of an expert layer: the residual's addition and
// the root-mean-square norm, to rows of the input's type and to 8-bit
// microscaled rows, and the gradients.  See include/ebc.h.
#include "ebc_mx8.cuh"

using namespace ebc;

namespace {

constexpr int kMaxThreads = 512;
constexpr int kRowThreads = 256;   // of a CTA whose rows take a warp or less each

// ---- one row on a group of threads ----
// A thread has N vectors of V consecutive values: vector n * lanes + its place
// in the group.  kLanes: the lanes of a warp that a row takes; 0: the whole CTA.

// The group's sums of K values a thread, the same in all its threads.  `part`
// has room for two rows, so one barrier a row is enough.
template <int kLanes, int K>
__device__ __forceinline__ void group_sum(float (&v)[K], float (*part)[K][kMaxThreads / 32], int turn) {
#pragma unroll
  for (int off = (kLanes ? kLanes : 32) / 2; off > 0; off >>= 1)
#pragma unroll
    for (int k = 0; k < K; ++k) v[k] += __shfl_xor_sync(0xffffffffu, v[k], off);
  if constexpr (kLanes == 0) {
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, warps = blockDim.x >> 5;
    if (lane == 0)
#pragma unroll
      for (int k = 0; k < K; ++k) part[turn][k][w] = v[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
      float s = lane < warps ? part[turn][k][lane] : 0.f;
#pragma unroll
      for (int off = kMaxThreads / 64; off > 0; off >>= 1) s += __shfl_xor_sync(0xffffffffu, s, off);
      v[k] = __shfl_sync(0xffffffffu, s, 0);
    }
  }
}

// V weights from the i-th on, of the type that the caller keeps them in.
template <int V>
__device__ __forceinline__ void load_weights(const void* w, int type, int64_t i, float (&f)[V]) {
  auto get = [&](auto one) {
    using W = decltype(one);
    Values<W, V> v;
    v.load((const W*)w + i);
#pragma unroll
    for (int k = 0; k < V; ++k) f[k] = to_f32(v.e[k]);
  };
  if (type == EBC_F32)
    get(float());
  else if (type == EBC_BF16)
    get(__nv_bfloat16());
  else
    get(__half());
}

struct NormArgs {
  const void *x, *r, *w;   // r: null without a residual
  void *y, *h;             // null where not asked for
  uint8_t *codes, *scales;
  Glob* glob;
  int64_t ld_x, ld_r, rows;
  int width, w_type;
  float eps;
};

// h = x + r, y = h / sqrt(mean(h^2) + eps) * w, in 32 bits: h is rounded once, to
// be kept, and y is of the sum before that rounding, rounded once to its type
// and once to 8 bits.
// Every input is read once and every output written once; bound by bandwidth.
template <typename T, int V, int N, int kLanes>
__global__ void __launch_bounds__(kMaxThreads) k_norm(NormArgs a) {
  __shared__ float part[2][1][kMaxThreads / 32];
  pdl_enter();
  const int lanes = kLanes ? kLanes : blockDim.x, at = threadIdx.x % lanes, groups = blockDim.x / lanes;
  const int64_t step = (int64_t)gridDim.x * groups;
  const int padded = (a.width + 31) / 32 * 32;
  const float share = 1.f / (float)a.width;
  int turn = 0;
  // the groups of a warp, and the warps of a CTA, go through the same rounds
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + threadIdx.x / lanes;
    const bool live = row < a.rows;
    Values<T, V> xv[N], rv[N];
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * lanes + at) * V;
      if (live && c < a.width) {
        xv[n].load((const T*)a.x + row * a.ld_x + c);
        if (a.r) rv[n].load((const T*)a.r + row * a.ld_r + c);
      } else {
        xv[n].zero();
        rv[n].zero();
      }
    }
    float f[N][V], sum[1] = {0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * lanes + at) * V;
      Values<T, V> hv;
#pragma unroll
      for (int k = 0; k < V; ++k) {
        f[n][k] = to_f32(xv[n].e[k]);
        if (a.r) f[n][k] += to_f32(rv[n].e[k]);
        hv.e[k] = from_f32<T>(f[n][k]);
        sum[0] += f[n][k] * f[n][k];
      }
      if (a.h && live && c < a.width) hv.store((T*)a.h + row * a.width + c);
    }
    group_sum<kLanes>(sum, part, turn);
    const float scale = rsqrtf(sum[0] * share + a.eps);
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * lanes + at) * V;
      if (c < a.width) {
        float w[V];
        load_weights<V>(a.w, a.w_type, c, w);
#pragma unroll
        for (int k = 0; k < V; ++k) f[n][k] = f[n][k] * scale * w[k];
      }
      if (a.y && live && c < a.width) {
        Values<T, V> yv;
#pragma unroll
        for (int k = 0; k < V; ++k) yv.e[k] = from_f32<T>(f[n][k]);
        yv.store((T*)a.y + row * a.width + c);
      }
      if (a.codes) {
        const uint32_t s = mx8_scale(mx8_block_max<V>(f[n]));   // (values past the row's end are zero)
        if (live && c < padded) {
          mx8_store<V>(f[n], s, a.codes + row * padded + c);
          if (c % 32 == 0) a.scales[row * EBC_MX8_SCALE_BYTES(a.width) + c / 32] = (uint8_t)s;
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
  static __device__ __forceinline__ void commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
  static __device__ __forceinline__ void wait() {   // for all but the latest kStages - 1
    asm volatile("cp.async.wait_group %0;" ::"n"(kStages - 1) : "memory");
  }
  static size_t bytes(int threads) { return (size_t)kStages * kStreams * N * kParts * 16 * threads; }
};

// With u = h / sqrt(mean(h^2) + eps) and q = dy * w:
//   dx = (q - u * mean(q * u)) / sqrt(mean(h^2) + eps) + dh,   dw = sum over rows of dy * u.
// Both means of a row come out of one pass over it.  A thread keeps the same
// columns in every row, and with them their part of dw, so dw takes one
// partial row a CTA, which k_norm_dweight adds up in a fixed order.
// Bound by bandwidth, if loads are in flight while a row's sums go around the
// CTA: with kStages, the rows to come are copied to shared memory meanwhile.
template <typename T, int V, int N, int kLanes, int kStages>
__global__ void __launch_bounds__(kLanes ? kRowThreads : kMaxThreads) k_norm_grad(GradArgs a) {
  using R = Ring<T, V, N, kStages>;
  __shared__ float part[2][2][kMaxThreads / 32];
  pdl_enter();
  const int lanes = kLanes ? kLanes : blockDim.x, at = threadIdx.x % lanes, groups = blockDim.x / lanes;
  const int64_t step = (int64_t)gridDim.x * groups;
  const float share = 1.f / (float)a.width;
  constexpr bool kKeep = N * V <= 16;   // the weights stay in registers
  float dw[N][V], kept[kKeep ? N : 1][V];
#pragma unroll
  for (int n = 0; n < N; ++n) {
#pragma unroll
    for (int k = 0; k < V; ++k) dw[n][k] = 0.f;
    if constexpr (kKeep) {
      const int c = (n * lanes + at) * V;
#pragma unroll
      for (int k = 0; k < V; ++k) kept[n][k] = 0.f;
      if (c < a.width) load_weights<V>(a.w, a.w_type, c, kept[n]);
    }
  }
  auto weights = [&](int n, int c, float (&w)[V]) {
    if constexpr (kKeep) {
#pragma unroll
      for (int k = 0; k < V; ++k) w[k] = kept[n][k];
    } else {
      load_weights<V>(a.w, a.w_type, c, w);
    }
  };
  auto request = [&](int64_t row, int stage) {
    if constexpr (kStages > 0) {
      if (row < a.rows) {
#pragma unroll
        for (int n = 0; n < N; ++n) {
          const int c = (n * lanes + at) * V;
          if (c >= a.width) continue;
          R::copy(stage, 0, n, (const T*)a.h + row * a.ld_h + c);
          R::copy(stage, 1, n, (const T*)a.dy + row * a.ld_dy + c);
          if (a.dh) R::copy(stage, 2, n, (const T*)a.dh + row * a.ld_dh + c);
        }
      }
      R::commit();
    }
  };
  int turn = 0, stage = 0;
  for (int i = 0; i < kStages - 1; ++i) request((int64_t)blockIdx.x * groups + i * step, i);
  for (int64_t row0 = (int64_t)blockIdx.x * groups; row0 < a.rows; row0 += step, turn ^= 1) {
    const int64_t row = row0 + threadIdx.x / lanes;
    const bool live = row < a.rows;
    Values<T, V> hv[N], gv[N], ev[N];
    if constexpr (kStages > 0) {
      request(row0 + (kStages - 1) * step, stage == 0 ? kStages - 1 : stage - 1);
      R::wait();
    }
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * lanes + at) * V;
      if (live && c < a.width) {
        if constexpr (kStages > 0) {
          R::get(stage, 0, n, &hv[n]);
          R::get(stage, 1, n, &gv[n]);
        } else {
          hv[n].load((const T*)a.h + row * a.ld_h + c);
          gv[n].load((const T*)a.dy + row * a.ld_dy + c);
          if (a.dh) ev[n].load((const T*)a.dh + row * a.ld_dh + c);
        }
      } else {
        hv[n].zero();
        gv[n].zero();
      }
    }
    float sum[2] = {0.f, 0.f};
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * lanes + at) * V;
      if (c >= a.width) continue;
      float w[V];
      weights(n, c, w);
#pragma unroll
      for (int k = 0; k < V; ++k) {
        const float h = to_f32(hv[n].e[k]);
        sum[0] += h * h;
        sum[1] += to_f32(gv[n].e[k]) * w[k] * h;
      }
    }
    group_sum<kLanes>(sum, part, turn);
    const float scale = rsqrtf(sum[0] * share + a.eps), mean = sum[1] * share * scale;
    if (live) {
#pragma unroll
      for (int n = 0; n < N; ++n) {
        const int c = (n * lanes + at) * V;
        if (c >= a.width) continue;
        float w[V];
        weights(n, c, w);
        Values<T, V> out;
        if constexpr (kStages > 0)
          if (a.dh) R::get(stage, 2, n, &ev[n]);
#pragma unroll
        for (int k = 0; k < V; ++k) {
          const float u = to_f32(hv[n].e[k]) * scale, g = to_f32(gv[n].e[k]);
          float d = scale * (g * w[k] - u * mean);
          if (a.dh) d += to_f32(ev[n].e[k]);
          out.e[k] = from_f32<T>(d);
          dw[n][k] += g * u;
        }
        out.store((T*)a.dx + row * a.width + c);
      }
    }
    if (++stage >= kStages) stage = 0;
  }
  float* mine = a.parts + (int64_t)blockIdx.x * a.width;
  if constexpr (kLanes == 0) {
#pragma unroll
    for (int n = 0; n < N; ++n) {
      const int c = (n * lanes + at) * V;
      if (c >= a.width) continue;
      if (gridDim.x == 1) {   // nothing to add up
#pragma unroll
        for (int k = 0; k < V; ++k) store_dweight(a.dw, a.w_type, c + k, dw[n][k]);
        continue;
      }
      Values<float, V> out;
#pragma unroll
      for (int k = 0; k < V; ++k) out.e[k] = dw[n][k];
      out.store(mine + c);
    }
  } else {
    // the CTA's groups one after the other, so that the order is the same in every run
    __shared__ float all[N * V * kLanes];
    for (int g = 0; g < groups; ++g) {
      if ((int)threadIdx.x / lanes == g)
#pragma unroll
        for (int n = 0; n < N; ++n)
#pragma unroll
          for (int k = 0; k < V; ++k) {
            float* p = all + (n * lanes + at) * V + k;
            *p = g ? *p + dw[n][k] : dw[n][k];
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

// A row's layout: values of a vector, vectors of a thread, lanes of a row (0: a
// CTA), threads of a CTA.
template <typename T_, int V_, int N_, int kLanes_>
struct Layout {
  using T = T_;
  static constexpr int V = V_, N = N_, kLanes = kLanes_;
};

// Calls f with the layout and the CTA's threads: a row on as few lanes as hold
// it with one vector each, then on more vectors a lane, then on a CTA.
template <typename T, typename F>
cudaError_t with_layout(int v, int width, F&& f) {
  auto cta = [&](auto layout) {
    const int each = layout.V * layout.N;
    return f(layout, ((width + each - 1) / each + 31) / 32 * 32);
  };
  if (v == 8) {
    if (width <= 64) return f(Layout<T, 8, 1, 8>{}, kRowThreads);
    if (width <= 128) return f(Layout<T, 8, 1, 16>{}, kRowThreads);
    if (width <= 256) return f(Layout<T, 8, 1, 32>{}, kRowThreads);
    if (width <= 512) return f(Layout<T, 8, 2, 32>{}, kRowThreads);
    if (width <= 2048) return cta(Layout<T, 8, 1, 0>{});
    if (width <= 8192) return cta(Layout<T, 8, 2, 0>{});
    return cta(Layout<T, 8, 4, 0>{});
  }
  if (v == 2) {
    if (width <= 512) return f(Layout<T, 2, 8, 32>{}, kRowThreads);
    if (width <= 4096) return cta(Layout<T, 2, 4, 0>{});
    return cta(Layout<T, 2, 16, 0>{});
  }
  if (width <= 256) return f(Layout<T, 1, 8, 32>{}, kRowThreads);
  if (width <= 4096) return cta(Layout<T, 1, 8, 0>{});
  return cta(Layout<T, 1, 32, 0>{});
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

// 8, 2 or 1 values that one access takes everywhere
int values_of(uintptr_t rows, int elem, const void* w, int w_elem) {
  const int a = row_values(rows, elem), b = row_values((uintptr_t)w, w_elem);
  return a < b ? a : b;
}

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
  const NormArgs a{d_x, d_residual, d_weight, d_y, d_h, d_codes, d_scales, v.glob, ld_x, ld_residual, rows,
                   (int)width, weight_type, eps};
  const int vals = values_of((uintptr_t)d_x | (uintptr_t)(ld_x * b) | (uintptr_t)(width * b) | (uintptr_t)d_y |
                                 (uintptr_t)d_h | (d_residual ? (uintptr_t)d_residual | (uintptr_t)(ld_residual * b) : 0),
                             b, d_weight, wb);
  return cuda_code(with_type_of(type, [&](auto one) {
    return with_layout<decltype(one)>(vals, (int)width, [&](auto l, int threads) {
      using L = decltype(l);
      const int groups = L::kLanes ? threads / L::kLanes : 1;
      const int64_t want = (rows + groups - 1) / groups, most = (int64_t)v.nsm * (2048 / threads) * 2;
      return launch_named(v, "k_norm", st, k_norm<typename L::T, L::V, L::N, L::kLanes>,
                          dim3((unsigned)(want < most ? want : most)), dim3(threads), 0, 1, a);
    });
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
    const int vals = values_of((uintptr_t)d_dy | (uintptr_t)(ld_dy * b) | (uintptr_t)d_h | (uintptr_t)(ld_h * b) |
                                   (uintptr_t)d_dx | (uintptr_t)(width * b) |
                                   (d_dh ? (uintptr_t)d_dh | (uintptr_t)(ld_dh * b) : 0),
                               b, d_weight, wb);
    // (fp32 partial rows start where the scratch's 16 bytes allow: whole vectors of 8 want 32)
    const int vals_s = row_values((uintptr_t)d_scratch | (uintptr_t)(width * 4), 4);
    e = with_type_of(type, [&](auto one) {
      return with_layout<decltype(one)>(vals < vals_s ? vals : vals_s, (int)width, [&](auto l, int threads) {
        using L = decltype(l);
        // A row a CTA of whole vectors: rows to come in shared memory, as many as
        // two CTAs an SM have room for.
        constexpr int kBytes = 3 * L::N * L::V * (int)sizeof(typename L::T) * kMaxThreads;
        constexpr int kStages = L::kLanes || L::V < 8 ? 0 : kBytes <= 48 * 1024 ? 4 : kBytes <= 96 * 1024 ? 2 : 0;
        const auto kernel = k_norm_grad<typename L::T, L::V, L::N, L::kLanes, kStages>;
        size_t smem = 0;
        if constexpr (kStages > 0) {
          using R = Ring<typename L::T, L::V, L::N, kStages>;
          const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                     (int)R::bytes(kMaxThreads));
          if (e != cudaSuccess) return e;
          smem = R::bytes(threads);
        }
        const int groups = L::kLanes ? threads / L::kLanes : 1;
        const int64_t want = (rows + groups - 1) / groups;
        // all CTAs at once: by their registers (at most 128 a thread) and shared memory
        constexpr int kFit = L::N * L::V <= 8 ? 1024 : 512;
        int64_t each = kFit / threads < 1 ? 1 : kFit / threads;
        if (smem && each > (int64_t)((220 * 1024) / (smem + 2048))) each = (int64_t)((220 * 1024) / (smem + 2048));
        int64_t most = (int64_t)v.nsm * (each < 1 ? 1 : each);
        if (most > EBC_NORM_GRAD_PARTS) most = EBC_NORM_GRAD_PARTS;
        a.n_parts = (int)(want < most ? want : most);
        return launch_named(v, "k_norm_grad", st, kernel, dim3((unsigned)a.n_parts), dim3(threads), smem, 1, a);
      });
    });
  }
  if (e == cudaSuccess && a.n_parts != 1)
    e = launch_named(v, "k_norm_dweight", st, k_norm_dweight, dim3((unsigned)((width + 31) / 32)), dim3(1024), 0, 1,
                     d_scratch, a.n_parts, (int)width, weight_type, d_dweight);
  return cuda_code(e);
}

}  // extern "C"
