// ebc_experts.cu -- tokens sorted by expert and back: the plan of a routed
// batch, the dispatch of its rows into a sending buffer that holds every
// expert's rows together, the weighted sum on the way back, and both
// gradients.  See include/ebc.h for the operators' definitions.
#include <cooperative_groups.h>

#include "ebc_types.cuh"

using namespace ebc;
namespace cg = cooperative_groups;

namespace {

constexpr int kPlanThreads = 1024;
constexpr int kPlanWarps = kPlanThreads / 32;

template <typename Id>
__device__ __forceinline__ int read_id(const Id* ids, int64_t s, int64_t n, int E, bool* bad) {
  if (s >= n) return -1;
  const Id v = ids[s];
  if (v >= (Id)E) *bad = true;
  return v >= 0 && v < (Id)E ? (int)v : -1;
}

// Stable counting sort of the n slots by expert, in one launch of one cluster.
//
// The slots are split evenly among the cluster's warps, in order.  Each warp
// counts its slots per expert (lanes of equal expert found with one match per
// 32 slots); the counts become, per warp and expert, the first row of that
// warp's slots (a scan over the warps of a CTA in shared memory, over the CTAs
// through distributed shared memory, over the experts by one thread each);
// then each warp walks its slots again and hands out rows.  No atomics on
// shared counters decide an order, so the plan is the same in every run.
//
// Bound by latency: the ids are read twice (the second time from L1/L2) and
// two ints a slot are written, far below a microsecond of bandwidth at
// 65,536 slots.
template <typename Id>
__global__ void __launch_bounds__(kPlanThreads) k_moe_plan(const Id* __restrict__ ids, int64_t n, int E,
                                                           int32_t* __restrict__ rows, int32_t* __restrict__ place,
                                                           int32_t* __restrict__ offsets, Glob* glob) {
  extern __shared__ uint32_t sm[];
  uint32_t* hist = sm;                        // [warps][E]
  uint32_t* total = sm + kPlanWarps * E;      // [E] this CTA's slots per expert
  __shared__ uint32_t s_warp[kPlanWarps];
  __shared__ uint32_t s_live;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
  for (int i = tid; i < kPlanWarps * E; i += kPlanThreads) hist[i] = 0u;
  pdl_enter();
  __syncthreads();

  const int64_t warps = (int64_t)C * kPlanWarps;
  const int64_t share = ((n + warps - 1) / warps + 31) & ~(int64_t)31;
  const int64_t first = ((int64_t)c * kPlanWarps + w) * share;
  const int64_t last = first + share < n ? first + share : n;
  uint32_t* mine = hist + w * E;
  bool bad = false;
  for (int64_t s = first; s < last; s += 32) {
    const int e = read_id(ids, s + lane, n, E, &bad);
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += (uint32_t)__popc(same);
    __syncwarp();
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(glob, EBC_ERR_INVALID_ARG);
  __syncthreads();
  // counts -> slots of the warps before, per expert
  if (tid < E) {
    uint32_t run = 0;
    for (int i = 0; i < kPlanWarps; ++i) {
      const uint32_t v = hist[i * E + tid];
      hist[i * E + tid] = run;
      run += v;
    }
    total[tid] = run;
  }
  cluster.sync();
  // over the CTAs, then over the experts
  uint32_t before = 0, all = 0;
  if (tid < E)
    for (int i = 0; i < C; ++i) {
      const uint32_t v = cluster.map_shared_rank(total, i)[tid];
      if (i < c) before += v;
      all += v;
    }
  uint32_t inc = all;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const uint32_t v = __shfl_up_sync(0xffffffffu, inc, off);
    if (lane >= off) inc += v;
  }
  if (lane == 31) s_warp[w] = inc;
  __syncthreads();
  uint32_t pre = 0;
  for (int i = 0; i < w; ++i) pre += s_warp[i];
  const uint32_t start = pre + inc - all;
  if (tid < E) {
    if (c == 0) offsets[tid] = (int32_t)start;
    const uint32_t base = start + before;
    for (int i = 0; i < kPlanWarps; ++i) hist[i * E + tid] += base;
  }
  if (tid == E - 1) {
    s_live = start + all;
    if (c == 0) offsets[E] = (int32_t)(start + all);
  }
  cluster.sync();   // the totals have been read; hist and s_live are complete
  for (int64_t s = first; s < last; s += 32) {
    bool ignore = false;
    const int e = read_id(ids, s + lane, n, E, &ignore);
    const unsigned same = __match_any_sync(0xffffffffu, e);
    if (e >= 0) {
      const uint32_t r = mine[e] + (uint32_t)__popc(same & ((1u << lane) - 1u));
      place[s + lane] = (int32_t)r;
      rows[r] = (int32_t)(s + lane);
    } else if (s + lane < n) {
      place[s + lane] = -1;
    }
    __syncwarp();
    if (e >= 0 && lane == __ffs(same) - 1) mine[e] += (uint32_t)__popc(same);
    __syncwarp();
  }
  for (int64_t r = (int64_t)s_live + (int64_t)c * kPlanThreads + tid; r < n; r += (int64_t)C * kPlanThreads)
    rows[r] = -1;
}

// The row of slot s, or -1 where it was dropped.  A row outside the buffer is
// an error of the caller's plan: recorded, and treated as dropped.
__device__ __forceinline__ int32_t read_place(const int32_t* place, int64_t s, int64_t n, Glob* glob) {
  const int32_t p = place[s];
  if (p >= n) record_error(glob, EBC_ERR_INVALID_ARG);
  return p >= 0 && p < n ? p : -1;
}

__device__ __forceinline__ int64_t live_rows(const int32_t* offsets, int E, int64_t n) {
  const int64_t v = offsets[E];
  return v < 0 ? 0 : v < n ? v : n;
}

constexpr int kRowWarps = 8;
constexpr int kScatterU = 4;   // vectors a lane holds of one piece of a row

// xs[place[t, j]] = x[t]: a warp takes a piece of a token's row (kScatterU
// vectors a lane), reads it once and writes it to every choice's row, so x is
// read once from memory.  Rows past the last expert's become zero.
// Bound by the bandwidth of the writes.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kRowWarps) k_moe_dispatch(const T* __restrict__ x, int64_t ld, int64_t tokens,
                                                                 int top, int64_t width,
                                                                 const int32_t* __restrict__ place,
                                                                 const int32_t* __restrict__ offsets, int E,
                                                                 T* __restrict__ xs, Glob* glob) {
  pdl_enter();
  using R = Vec<T, V>;
  constexpr int kPiece = 32 * kScatterU * R::kN;   // elements of a piece
  const int lane = threadIdx.x & 31;
  const int64_t n = tokens * top, pieces = (width + kPiece - 1) / kPiece;
  const int64_t live = live_rows(offsets, E, n);
  const int64_t units = (tokens + (n - live)) * pieces;
  for (int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kRowWarps) {
    const int64_t t = u / pieces, h0 = (u - t * pieces) * kPiece + lane * R::kN;
    R v[kScatterU];
    if (t < tokens) {
      const T* src = x + t * ld;
#pragma unroll
      for (int i = 0; i < kScatterU; ++i) {
        const int64_t h = h0 + (int64_t)i * 32 * R::kN;
        if (h < width) v[i].raw = *reinterpret_cast<const typename Raw<V>::T*>(src + h);
      }
      for (int j0 = 0; j0 < top; j0 += 32) {
        const int m = top - j0 < 32 ? top - j0 : 32;
        const int32_t p_lane = lane < m ? read_place(place, t * top + j0 + lane, n, glob) : -1;
        for (int j = 0; j < m; ++j) {
          const int32_t p = __shfl_sync(0xffffffffu, p_lane, j);
          if (p < 0) continue;
          T* dst = xs + (int64_t)p * width;
#pragma unroll
          for (int i = 0; i < kScatterU; ++i) {
            const int64_t h = h0 + (int64_t)i * 32 * R::kN;
            if (h < width) *reinterpret_cast<typename Raw<V>::T*>(dst + h) = v[i].raw;
          }
        }
      }
    } else {
      T* dst = xs + (live + (t - tokens)) * width;
#pragma unroll
      for (int k = 0; k < R::kN; ++k) v[0].e[k] = from_f32<T>(0.f);
#pragma unroll
      for (int i = 0; i < kScatterU; ++i) {
        const int64_t h = h0 + (int64_t)i * 32 * R::kN;
        if (h < width) *reinterpret_cast<typename Raw<V>::T*>(dst + h) = v[0].raw;
      }
    }
  }
}

// y[t] = sum over j of w[t, j] * ys[place[t, j]] (weights null: 1), held in
// fp32 and added in the order of j; a dropped choice adds nothing, whatever
// its weight.  A warp takes one vector a lane of a token's row, four rows'
// loads in flight.  Bound by the bandwidth of the reads.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kRowWarps) k_moe_combine(const T* __restrict__ ys, int64_t ld, int64_t tokens,
                                                                int top, int64_t width,
                                                                const int32_t* __restrict__ place,
                                                                const float* __restrict__ weights, T* __restrict__ y,
                                                                Glob* glob) {
  pdl_enter();
  using R = Vec<T, V>;
  constexpr int kPiece = 32 * R::kN;
  const int lane = threadIdx.x & 31;
  const int64_t n = tokens * top, pieces = (width + kPiece - 1) / kPiece, units = tokens * pieces;
  for (int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kRowWarps) {
    const int64_t t = u / pieces, h = (u - t * pieces) * kPiece + lane * R::kN;
    float acc[R::kN];
#pragma unroll
    for (int k = 0; k < R::kN; ++k) acc[k] = 0.f;
    for (int j0 = 0; j0 < top; j0 += 32) {
      const int m = top - j0 < 32 ? top - j0 : 32;
      const int64_t s = t * top + j0 + lane;
      const int32_t p_lane = lane < m ? read_place(place, s, n, glob) : -1;
      const float w_lane = lane < m && weights ? weights[s] : 1.f;
      for (int j = 0; j < m; j += 4) {
        R v[4];
        int32_t p[4];
        float w[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          p[i] = __shfl_sync(0xffffffffu, p_lane, (j + i) & 31);
          w[i] = __shfl_sync(0xffffffffu, w_lane, (j + i) & 31);
          if (j + i >= m) p[i] = -1;
          if (p[i] >= 0 && h < width)
            v[i].raw = *reinterpret_cast<const typename Raw<V>::T*>(ys + (int64_t)p[i] * ld + h);
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (p[i] >= 0 && h < width)
#pragma unroll
            for (int k = 0; k < R::kN; ++k) acc[k] = fmaf(w[i], to_f32(v[i].e[k]), acc[k]);
      }
    }
    if (h < width) {
      R o;
#pragma unroll
      for (int k = 0; k < R::kN; ++k) o.e[k] = from_f32<T>(acc[k]);
      *reinterpret_cast<typename Raw<V>::T*>(y + t * width + h) = o.raw;
    }
  }
}

// One slot a warp: dys[p] = w * dy[t] and dw = <dy[t], ys[p]> in one pass over
// the two rows (dy[t] comes from L1 or L2 for all but the first of a token's
// choices).  The dot product is held in fp32: per lane in the order of the
// row, then over the lanes by a fixed tree.  Rows past the last expert's
// become zero.  Bound by bandwidth.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kRowWarps) k_moe_combine_grad(
    const T* __restrict__ dy, int64_t ld_dy, const T* __restrict__ ys, int64_t ld_ys, int64_t tokens, int top,
    int64_t width, const int32_t* __restrict__ place, const int32_t* __restrict__ offsets, int E,
    const float* __restrict__ weights, T* __restrict__ dys, float* __restrict__ dw, Glob* glob) {
  pdl_enter();
  using R = Vec<T, V>;
  constexpr int kStep = 32 * R::kN;
  const int lane = threadIdx.x & 31;
  const int64_t n = tokens * top;
  const int64_t live = live_rows(offsets, E, n);
  const int64_t units = n + (n - live);
  for (int64_t s = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); s < units;
       s += (int64_t)gridDim.x * kRowWarps) {
    if (s >= n) {
      T* dst = dys + (live + (s - n)) * width;
      R z;
#pragma unroll
      for (int k = 0; k < R::kN; ++k) z.e[k] = from_f32<T>(0.f);
      for (int64_t h = lane * R::kN; h < width; h += kStep) *reinterpret_cast<typename Raw<V>::T*>(dst + h) = z.raw;
      continue;
    }
    const int32_t p = read_place(place, s, n, glob);
    if (p < 0) {
      if (lane == 0) dw[s] = 0.f;
      continue;
    }
    const float w = weights[s];
    const T* a = dy + (s / top) * ld_dy;
    const T* b = ys + (int64_t)p * ld_ys;
    T* dst = dys + (int64_t)p * width;
    float dot = 0.f;
#pragma unroll 4
    for (int64_t h = lane * R::kN; h < width; h += kStep) {
      R va, vb, o;
      va.raw = *reinterpret_cast<const typename Raw<V>::T*>(a + h);
      vb.raw = *reinterpret_cast<const typename Raw<V>::T*>(b + h);
#pragma unroll
      for (int k = 0; k < R::kN; ++k) {
        const float g = to_f32(va.e[k]);
        dot = fmaf(g, to_f32(vb.e[k]), dot);
        o.e[k] = from_f32<T>(w * g);
      }
      *reinterpret_cast<typename Raw<V>::T*>(dst + h) = o.raw;
    }
#pragma unroll
    for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    if (lane == 0) dw[s] = dot;
  }
}

// CTAs for `units` warps of work: one warp each up to 16 resident CTAs a SM in
// 8 turns; the kernels loop beyond that.
unsigned row_grid(int64_t units, int nsm) {
  const int64_t want = (units + kRowWarps - 1) / kRowWarps, most = (int64_t)nsm * 16 * 8;
  return (unsigned)(want < 1 ? 1 : want < most ? want : most);
}

bool routed_ok(int64_t tokens, int top, int n_experts) {
  return tokens >= 0 && top >= 1 && top <= EBC_MAX_EXPERTS && n_experts >= 1 && n_experts <= EBC_MAX_EXPERTS &&
         tokens <= (int64_t)INT32_MAX / top;
}

bool rows_ok(int type, int64_t width, int64_t ld) {
  return type_bytes(type) != 0 && width >= 1 && width <= (1 << 24) && ld >= width && ld <= ((int64_t)1 << 40);
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

template <typename Id>
cudaError_t plan_t(const CallView& v, const Id* ids, int64_t n, int E, int32_t* rows, int32_t* place,
                   int32_t* offsets, cudaStream_t st) {
  const size_t smem = sizeof(uint32_t) * (size_t)(kPlanWarps + 1) * E;
  if (smem > 48 * 1024) {
    const cudaError_t e =
        cudaFuncSetAttribute(k_moe_plan<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
  }
  const unsigned C = n <= 4096 ? 1 : 8;
  return launch_named(v, "k_moe_plan", st, k_moe_plan<Id>, dim3(C), dim3(kPlanThreads), smem, C, ids, n, E, rows,
                      place, offsets, v.glob);
}

}  // namespace

extern "C" {

int ebc_moe_plan(ebc_ctx* ctx, const void* d_ids, int id_bytes, int64_t tokens, int top, int n_experts,
                 int32_t* d_rows, int32_t* d_place, int32_t* d_offsets, void* stream) {
  if (!ctx || !routed_ok(tokens, top, n_experts) || (id_bytes != 4 && id_bytes != 8) || !d_offsets ||
      !aligned(d_offsets, 4))
    return EBC_ERR_INVALID_ARG;
  if (tokens > 0 && (!d_ids || !aligned(d_ids, id_bytes) || !d_rows || !aligned(d_rows, 4) || !d_place ||
                     !aligned(d_place, 4)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc) return rc;
  const int64_t n = tokens * top;
  return cuda_code(id_bytes == 4 ? plan_t(v, (const int32_t*)d_ids, n, n_experts, d_rows, d_place, d_offsets, st)
                                 : plan_t(v, (const int64_t*)d_ids, n, n_experts, d_rows, d_place, d_offsets, st));
}

int ebc_moe_dispatch(ebc_ctx* ctx, const void* d_x, int64_t ld_x, int type, int64_t tokens, int top, int64_t width,
                     const int32_t* d_place, const int32_t* d_offsets, int n_experts, void* d_xs, void* stream) {
  const int b = type_bytes(type);
  if (!ctx || !routed_ok(tokens, top, n_experts) || !rows_ok(type, width, ld_x) || !d_offsets ||
      !aligned(d_offsets, 4))
    return EBC_ERR_INVALID_ARG;
  if (tokens > 0 && (!d_x || !aligned(d_x, b) || !d_place || !aligned(d_place, 4) || !d_xs || !aligned(d_xs, b)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || tokens == 0) return rc;
  const int vb = vec_bytes((uintptr_t)d_x | (uintptr_t)d_xs | (uintptr_t)(ld_x * b) | (uintptr_t)(width * b), b);
  return cuda_code(with_type(type, vb, [&](auto tag) {
    using T = typename decltype(tag)::T;
    constexpr int V = decltype(tag)::V;
    const int64_t piece = 32 * kScatterU * (V / (int)sizeof(T));
    return launch_named(v, "k_moe_dispatch", st, k_moe_dispatch<T, V>,
                        dim3(row_grid(tokens * ((width + piece - 1) / piece), v.nsm)), dim3(32 * kRowWarps), 0, 1,
                        (const T*)d_x, ld_x, tokens, top, width, d_place, d_offsets, n_experts, (T*)d_xs, v.glob);
  }));
}

int ebc_moe_combine(ebc_ctx* ctx, const void* d_ys, int64_t ld_ys, int type, int64_t tokens, int top, int64_t width,
                    const int32_t* d_place, const float* d_weights, void* d_y, void* stream) {
  const int b = type_bytes(type);
  if (!ctx || !routed_ok(tokens, top, 1) || !rows_ok(type, width, ld_ys) || !aligned(d_weights, 4))
    return EBC_ERR_INVALID_ARG;
  if (tokens > 0 && (!d_ys || !aligned(d_ys, b) || !d_place || !aligned(d_place, 4) || !d_y || !aligned(d_y, b)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || tokens == 0) return rc;
  const int vb = vec_bytes((uintptr_t)d_ys | (uintptr_t)d_y | (uintptr_t)(ld_ys * b) | (uintptr_t)(width * b), b);
  return cuda_code(with_type(type, vb, [&](auto tag) {
    using T = typename decltype(tag)::T;
    constexpr int V = decltype(tag)::V;
    const int64_t piece = 32 * (V / (int)sizeof(T));
    return launch_named(v, "k_moe_combine", st, k_moe_combine<T, V>,
                        dim3(row_grid(tokens * ((width + piece - 1) / piece), v.nsm)), dim3(32 * kRowWarps), 0, 1,
                        (const T*)d_ys, ld_ys, tokens, top, width, d_place, d_weights, (T*)d_y, v.glob);
  }));
}

int ebc_moe_combine_grad(ebc_ctx* ctx, const void* d_dy, int64_t ld_dy, const void* d_ys, int64_t ld_ys, int type,
                         int64_t tokens, int top, int64_t width, const int32_t* d_place, const int32_t* d_offsets,
                         int n_experts, const float* d_weights, void* d_dys, float* d_dweights, void* stream) {
  const int b = type_bytes(type);
  if (!ctx || !routed_ok(tokens, top, n_experts) || !rows_ok(type, width, ld_dy) || !rows_ok(type, width, ld_ys) ||
      !d_offsets || !aligned(d_offsets, 4))
    return EBC_ERR_INVALID_ARG;
  if (tokens > 0 && (!d_dy || !aligned(d_dy, b) || !d_ys || !aligned(d_ys, b) || !d_place || !aligned(d_place, 4) ||
                     !d_weights || !aligned(d_weights, 4) || !d_dys || !aligned(d_dys, b) || !d_dweights ||
                     !aligned(d_dweights, 4)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || tokens == 0) return rc;
  const int vb = vec_bytes((uintptr_t)d_dy | (uintptr_t)d_ys | (uintptr_t)d_dys | (uintptr_t)(ld_dy * b) |
                               (uintptr_t)(ld_ys * b) | (uintptr_t)(width * b),
                           b);
  return cuda_code(with_type(type, vb, [&](auto tag) {
    using T = typename decltype(tag)::T;
    constexpr int V = decltype(tag)::V;
    return launch_named(v, "k_moe_combine_grad", st, k_moe_combine_grad<T, V>,
                        dim3(row_grid(tokens * top, v.nsm)), dim3(32 * kRowWarps), 0, 1, (const T*)d_dy, ld_dy,
                        (const T*)d_ys, ld_ys, tokens, top, width, d_place, d_offsets, n_experts, d_weights,
                        (T*)d_dys, d_dweights, v.glob);
  }));
}

}  // extern "C"
