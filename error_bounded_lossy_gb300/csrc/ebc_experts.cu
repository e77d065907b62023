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

constexpr int kPlanBatch = 8;   // rounds of 32 slots whose ids a warp has in flight

// Ids of up to kPlanBatch rounds from slot s on; -1 past the end and for what
// is no expert.
template <typename Id>
__device__ __forceinline__ void read_ids(const Id* ids, int64_t s, int64_t last, int E, int (&e)[kPlanBatch],
                                         bool* bad) {
  Id v[kPlanBatch];
#pragma unroll
  for (int i = 0; i < kPlanBatch; ++i) v[i] = s + 32 * i < last ? ids[s + 32 * i] : (Id)-1;
#pragma unroll
  for (int i = 0; i < kPlanBatch; ++i) {
    if (v[i] >= (Id)E) *bad = true;
    e[i] = v[i] >= 0 && v[i] < (Id)E ? (int)v[i] : -1;
  }
}

// The lanes of equal value, for values 0 .. 2^bits - 1: one vote a bit.  (The
// match instruction has the same answer and took 53 cycles a warp here, which
// made it most of the plan's time.)
__device__ __forceinline__ unsigned equal_lanes(int v, int bits) {
  unsigned same = 0xffffffffu;
  for (int b = 0; b < bits; ++b) {
    const unsigned set = __ballot_sync(0xffffffffu, (v >> b) & 1);
    same &= (v >> b) & 1 ? set : ~set;
  }
  return same;
}

// Stable counting sort of the n slots by expert, in one launch of one cluster.
//
// The slots are split evenly among the cluster's warps, in order.  Each warp
// counts its slots per expert (lanes of equal expert found by votes); the counts
// become, per warp and expert, the warp's first place among the expert's slots of
// its CTA (a scan over the warps), which the CTAs' totals (read through
// distributed shared memory) and a scan over the experts turn into rows; then
// each warp walks its slots again and hands out rows.  No atomics on shared
// counters decide an order, so the plan is the same in every run.
//
// Bound by latency: the ids are read once where a warp's share is one batch
// (else twice) and two ints a slot are written, far below a microsecond of
// bandwidth at 65,536 slots.
template <typename Id>
__global__ void __launch_bounds__(kPlanThreads) k_moe_plan(const Id* ids, int64_t n, int E,
                                                           int32_t* __restrict__ rows, int32_t* __restrict__ place,
                                                           int32_t* __restrict__ offsets, Glob* glob) {
  extern __shared__ uint32_t sm[];
  const int pitch = E | 1;                       // an odd stride: the warps' counts of an expert in 32 banks
  uint32_t* hist = sm;                           // [warps][pitch]
  uint32_t* total = sm + kPlanWarps * pitch;     // [E] this CTA's slots per expert
  uint32_t* base = total + E;                    // [E] first row of this CTA's slots of each expert
  __shared__ uint32_t s_warp[kPlanWarps];
  __shared__ uint32_t s_live;
  cg::cluster_group cluster = cg::this_cluster();
  const int tid = threadIdx.x, lane = tid & 31, w = tid >> 5;
  const int C = (int)cluster.num_blocks(), c = (int)cluster.block_rank();
  for (int i = tid; i < kPlanWarps * pitch; i += kPlanThreads) hist[i] = 0u;
  pdl_enter();

  const int64_t warps = (int64_t)C * kPlanWarps;
  const int64_t share = ((n + warps - 1) / warps + 31) & ~(int64_t)31;
  const int64_t first = ((int64_t)c * kPlanWarps + w) * share;
  const int64_t last = first + share < n ? first + share : n;
  constexpr int kStep = 32 * kPlanBatch;
  const bool once = share <= kStep;
  const int bits = 32 - __clz(E);   // of 0 (none) .. E
  uint32_t* mine = hist + w * pitch;
  bool bad = false;
  int e[kPlanBatch];
  read_ids(ids, first + lane, last, E, e, &bad);
  __syncthreads();   // the counts are zero
  for (int64_t s = first; s < last; s += kStep) {
    if (s > first) read_ids(ids, s + lane, last, E, e, &bad);
#pragma unroll
    for (int i = 0; i < kPlanBatch; ++i) {
      if (s + 32 * i >= last) break;
      const unsigned same = equal_lanes(e[i] + 1, bits);
      if (e[i] >= 0 && lane == __ffs(same) - 1) mine[e[i]] += (uint32_t)__popc(same);
      __syncwarp();
    }
  }
  if (__any_sync(0xffffffffu, bad) && lane == 0) record_error(glob, EBC_ERR_INVALID_ARG);
  __syncthreads();
  // counts -> slots of the warps before, a warp an expert and a lane a warp
  for (int x = w; x < E; x += kPlanWarps) {
    const uint32_t v = hist[lane * pitch + x];
    uint32_t inc = v;
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const uint32_t u = __shfl_up_sync(0xffffffffu, inc, off);
      if (lane >= off) inc += u;
    }
    hist[lane * pitch + x] = inc - v;
    if (lane == 31) total[x] = inc;
  }
  if (C > 1) cluster.sync(); else __syncthreads();
  // over the CTAs, then over the experts, a thread each
  uint32_t before = 0, all = 0;
  if (tid < E)
    for (int i = 0; i < C; ++i) {
      const uint32_t v = (C > 1 ? cluster.map_shared_rank(total, i) : total)[tid];
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
  uint32_t pre = lane < w ? s_warp[lane] : 0u;
  pre = __reduce_add_sync(0xffffffffu, pre);
  const uint32_t start = pre + inc - all;
  if (tid < E) {
    if (c == 0) offsets[tid] = (int32_t)start;
    base[tid] = start + before;
  }
  if (tid == E - 1) {
    s_live = start + all;
    if (c == 0) offsets[E] = (int32_t)(start + all);
  }
  if (C > 1) cluster.sync(); else __syncthreads();   // the totals have been read; base and s_live are complete
  for (int64_t s = first; s < last; s += kStep) {
    bool ignore = false;
    if (!once) read_ids(ids, s + lane, last, E, e, &ignore);
#pragma unroll
    for (int i = 0; i < kPlanBatch; ++i) {
      const int64_t at = s + 32 * i + lane;
      if (s + 32 * i >= last) break;
      const unsigned same = equal_lanes(e[i] + 1, bits);
      if (e[i] >= 0) {
        const uint32_t r = base[e[i]] + mine[e[i]] + (uint32_t)__popc(same & ((1u << lane) - 1u));
        place[at] = (int32_t)r;
        rows[r] = (int32_t)at;
      } else if (at < last) {
        place[at] = -1;
      }
      __syncwarp();
      if (e[i] >= 0 && lane == __ffs(same) - 1) mine[e[i]] += (uint32_t)__popc(same);
      __syncwarp();
    }
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

// a / b; most often in 32 bits, a fifth of the instructions
__device__ __forceinline__ int64_t divide(int64_t a, int64_t b) {
  return a <= UINT32_MAX ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// Vectors of V bytes a lane holds of one piece of a row.
template <int V>
constexpr int scatter_vectors() {
  return V >= 8 ? 4 : 8;
}

// xs[place[t, j]] = x[t]: a warp takes a piece of a token's row, reads it once and writes it to every choice's row, so x is
// read once from memory.  Rows past the last expert's become zero.
// Bound by the bandwidth of the writes.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kRowWarps) k_moe_dispatch(const T* x, int64_t ld, int64_t tokens,
                                                                 int top, int64_t width,
                                                                 const int32_t* place,
                                                                 const int32_t* offsets, int E,
                                                                 T* __restrict__ xs, Glob* glob) {
  pdl_enter();
  using R = Vec<T, V>;
  constexpr int kScatterU = scatter_vectors<V>(), kPiece = 32 * kScatterU * R::kN;   // elements of a piece
  const int lane = threadIdx.x & 31;
  const int64_t n = tokens * top, pieces = (width + kPiece - 1) / kPiece;
  const int64_t live = live_rows(offsets, E, n);
  const int64_t units = (tokens + (n - live)) * pieces;
  for (int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kRowWarps) {
    const int64_t t = divide(u, pieces), h0 = (u - t * pieces) * kPiece + lane * R::kN;
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

// The same for rows that are codes and scales: a row is code_vecs and scale_vecs
// vectors of 16 bytes, in two arrays.
__global__ void __launch_bounds__(32 * kRowWarps) k_moe_dispatch_mx(const uint4* codes, int64_t code_vecs,
                                                                    const uint4* scales, int64_t scale_vecs,
                                                                    int64_t tokens, int top, const int32_t* place,
                                                                    const int32_t* offsets, int E,
                                                                    uint4* __restrict__ xs_codes,
                                                                    uint4* __restrict__ xs_scales, Glob* glob) {
  pdl_enter();
  constexpr int kU = scatter_vectors<16>(), kPiece = 32 * kU;
  const int lane = threadIdx.x & 31;
  const int64_t n = tokens * top, vecs = code_vecs + scale_vecs, pieces = (vecs + kPiece - 1) / kPiece;
  const int64_t live = live_rows(offsets, E, n);
  const int64_t units = (tokens + (n - live)) * pieces;
  for (int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kRowWarps) {
    const int64_t t = divide(u, pieces), h0 = (u - t * pieces) * kPiece + lane;
    // a vector's place in both arrays' first rows, and from row to row
    const uint4* src[kU];
    uint4* dst[kU];
    int64_t hop[kU];
    uint4 v[kU];
#pragma unroll
    for (int i = 0; i < kU; ++i) {
      const int64_t h = h0 + i * 32;
      const bool code = h < code_vecs;
      hop[i] = h < vecs ? code ? code_vecs : scale_vecs : 0;   // 0: no vector
      src[i] = code ? codes + h : scales + (h - code_vecs);
      dst[i] = code ? xs_codes + h : xs_scales + (h - code_vecs);
    }
    auto store = [&](int64_t r) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (hop[i]) dst[i][r * hop[i]] = v[i];
    };
    if (t < tokens) {
#pragma unroll
      for (int i = 0; i < kU; ++i)
        if (hop[i]) v[i] = src[i][t * hop[i]];
      for (int j0 = 0; j0 < top; j0 += 32) {
        const int m = top - j0 < 32 ? top - j0 : 32;
        const int32_t p_lane = lane < m ? read_place(place, t * top + j0 + lane, n, glob) : -1;
        for (int j = 0; j < m; ++j) {
          const int32_t p = __shfl_sync(0xffffffffu, p_lane, j);
          if (p >= 0) store(p);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < kU; ++i) v[i] = make_uint4(0u, 0u, 0u, 0u);
      store(live + (t - tokens));
    }
  }
}

// Vectors of V bytes a lane takes of a row at a time (1 KB of a wide row a
// warp), and rows in flight.  Longer pieces of fewer rows suit the memory
// better than more rows at once: 8192 tokens x 8 choices x 4096 bf16 took
// 95 us so; 112 with 512 bytes of two rows, 125 of four, 189 of eight, and 134
// with 1 KB of four rows, 100 with 2 KB of one.
template <typename T, int V>
constexpr int gather_vectors() {
  constexpr int kN = V / (int)sizeof(T);
  return kN >= 4 ? 2 : 8 / kN;
}
constexpr int kGatherRows = 2;

// y[t] = sum over j of w[t, j] * ys[place[t, j]] (weights null: 1), held in
// fp32 and added in the order of j; a dropped choice adds nothing, whatever
// its weight.  A warp takes a piece of a token's row, kGatherRows rows' loads
// in flight.  Bound by the bandwidth of the reads.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kRowWarps) k_moe_combine(const T* ys, int64_t ld, int64_t tokens,
                                                                int top, int64_t width,
                                                                const int32_t* place,
                                                                const float* weights, T* __restrict__ y,
                                                                Glob* glob) {
  pdl_enter();
  using R = Vec<T, V>;
  constexpr int kU = gather_vectors<T, V>(), kStep = 32 * R::kN, kPiece = kU * kStep;
  const int lane = threadIdx.x & 31;
  const int64_t n = tokens * top;
  const int64_t pieces = (width + kPiece - 1) / kPiece, units = tokens * pieces;
  for (int64_t u = (int64_t)blockIdx.x * kRowWarps + (threadIdx.x >> 5); u < units;
       u += (int64_t)gridDim.x * kRowWarps) {
    const int64_t t = divide(u, pieces);
    const int64_t h = (u - t * pieces) * kPiece + lane * R::kN;
    const int left = (int)(width - h < kPiece ? width - h : kPiece);   // of the lane's values; may be <= 0
    float acc[kU][R::kN];
#pragma unroll
    for (int i = 0; i < kU; ++i)
#pragma unroll
      for (int k = 0; k < R::kN; ++k) acc[i][k] = 0.f;
    for (int j0 = 0; j0 < top; j0 += 32) {
      const int m = top - j0 < 32 ? top - j0 : 32;
      const int64_t s = t * top + j0 + lane;
      const int32_t p_lane = lane < m ? read_place(place, s, n, glob) : -1;
      const float w_lane = lane < m && weights ? weights[s] : 1.f;
      for (int j = 0; j < m; j += kGatherRows) {
        R v[kGatherRows][kU];
        int32_t p[kGatherRows];
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
          p[r] = __shfl_sync(0xffffffffu, p_lane, (j + r) & 31);
          if (j + r >= m) p[r] = -1;
          const T* src = ys + (int64_t)p[r] * ld + h;
          if (p[r] >= 0)
#pragma unroll
            for (int i = 0; i < kU; ++i)
              if (i * kStep < left) v[r][i].raw = *reinterpret_cast<const typename Raw<V>::T*>(src + i * kStep);
        }
#pragma unroll
        for (int r = 0; r < kGatherRows; ++r) {
          const float w = __shfl_sync(0xffffffffu, w_lane, (j + r) & 31);
          if (p[r] >= 0)
#pragma unroll
            for (int i = 0; i < kU; ++i)
              if (i * kStep < left)
#pragma unroll
                for (int k = 0; k < R::kN; ++k) acc[i][k] = fmaf(w, to_f32(v[r][i].e[k]), acc[i][k]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kU; ++i)
      if (i * kStep < left) {
        R o;
#pragma unroll
        for (int k = 0; k < R::kN; ++k) o.e[k] = from_f32<T>(acc[i][k]);
        *reinterpret_cast<typename Raw<V>::T*>(y + t * width + h + i * kStep) = o.raw;
      }
  }
}

// dys[p] = w * dy[t] and dw = <dy[t], ys[p]> in one pass over the two rows of a
// slot (dy[t] comes from L1 or L2 for all but the first of a token's choices).
// `split` warps of a CTA share a slot, so that few slots still fill the
// machine: 777 tokens x 3 choices x 1003 fp16 took 7.4 us with one warp each.
// The dot product is held in fp32: per lane in the order of the row, over the
// lanes by a fixed tree, then over the warps in order.  Rows past the last
// expert's become zero.  Bound by bandwidth.
template <typename T, int V>
__global__ void __launch_bounds__(32 * kRowWarps) k_moe_combine_grad(
    const T* dy, int64_t ld_dy, const T* ys, int64_t ld_ys, int64_t tokens, int top,
    int64_t width, const int32_t* place, const int32_t* offsets, int E,
    const float* weights, T* __restrict__ dys, float* __restrict__ dw, int split, Glob* glob) {
  __shared__ float s_dot[kRowWarps];
  pdl_enter();
  using R = Vec<T, V>;
  constexpr int kStep = 32 * R::kN, kU = R::kN >= 4 ? 4 : 8;   // vectors of each row in flight
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  const int part = w & (split - 1), slots = kRowWarps / split;
  const int64_t n = tokens * top;
  const int64_t live = live_rows(offsets, E, n);
  const int64_t units = n + (n - live);
  const int64_t h0 = (int64_t)part * kU * kStep + lane * R::kN, stride = (int64_t)split * kU * kStep;
  for (int64_t s0 = (int64_t)blockIdx.x * slots; s0 < units; s0 += (int64_t)gridDim.x * slots) {
    const int64_t s = s0 + w / split;
    const int32_t p = s < n ? read_place(place, s, n, glob) : -1;
    float dot = 0.f;
    if (p >= 0) {
      const float scale = weights[s];
      const T* a = dy + divide(s, top) * ld_dy + h0;
      const T* b = ys + (int64_t)p * ld_ys + h0;
      T* dst = dys + (int64_t)p * width + h0;
      for (int64_t left = width - h0; left > 0; left -= stride) {
        R va[kU], vb[kU];
#pragma unroll
        for (int i = 0; i < kU; ++i)
          if (i * kStep < left) {
            va[i].raw = *reinterpret_cast<const typename Raw<V>::T*>(a + i * kStep);
            vb[i].raw = *reinterpret_cast<const typename Raw<V>::T*>(b + i * kStep);
          }
#pragma unroll
        for (int i = 0; i < kU; ++i)
          if (i * kStep < left) {
            R o;
#pragma unroll
            for (int k = 0; k < R::kN; ++k) {
              const float g = to_f32(va[i].e[k]);
              dot = fmaf(g, to_f32(vb[i].e[k]), dot);
              o.e[k] = from_f32<T>(scale * g);
            }
            *reinterpret_cast<typename Raw<V>::T*>(dst + i * kStep) = o.raw;
          }
        a += stride;
        b += stride;
        dst += stride;
      }
#pragma unroll
      for (int off = 16; off; off >>= 1) dot += __shfl_xor_sync(0xffffffffu, dot, off);
    } else if (s >= n && s < units) {
      T* dst = dys + (live + (s - n)) * width;
      R z;
#pragma unroll
      for (int k = 0; k < R::kN; ++k) z.e[k] = from_f32<T>(0.f);
      for (int64_t h = (part * 32 + lane) * R::kN; h < width; h += split * kStep)
        *reinterpret_cast<typename Raw<V>::T*>(dst + h) = z.raw;
    }
    if (split > 1) {
      __syncthreads();   // the sums of the slots before have been read
      if (lane == 0) s_dot[w] = dot;
      __syncthreads();
      if (part == 0 && lane == 0)
        for (int i = 1; i < split; ++i) dot += s_dot[w + i];
    }
    if (part == 0 && lane == 0 && s < n) dw[s] = dot;
  }
}

// CTAs for `units` warps of work: a warp each, up to 128 CTAs a SM (16 turns of
// the 8 that are resident at once); the kernels loop beyond that.
unsigned row_grid(int64_t units, int nsm) {
  const int64_t want = (units + kRowWarps - 1) / kRowWarps, most = (int64_t)nsm * 8 * 16;
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

// Bytes of the plan's counts for E experts.
constexpr size_t plan_shared(int E) { return sizeof(uint32_t) * ((size_t)kPlanWarps * (E | 1) + 2 * (size_t)E); }

// Whether the device (or what this process may use of it) has a cluster of 16
// CTAs of the plan, whose size is not one that every device has.
template <typename Id>
cudaError_t ask_cluster(unsigned* most) {
  const cudaError_t e = cudaFuncSetAttribute(k_moe_plan<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                             (int)plan_shared(EBC_MAX_EXPERTS));
  if (e != cudaSuccess) return e;
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = 16;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(16);
  cfg.blockDim = dim3(kPlanThreads);
  cfg.dynamicSmemBytes = plan_shared(EBC_MAX_EXPERTS);
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  int clusters = 0;
  if (cudaOccupancyMaxActiveClusters(&clusters, k_moe_plan<Id>, &cfg) != cudaSuccess) {
    cudaGetLastError();   // "none" may be said so
    clusters = 0;
  }
  *most = clusters > 0 ? 16 : 8;
  return cudaSuccess;
}

template <typename Id>
cudaError_t plan_t(const CallView& v, const Id* ids, int64_t n, int E, int32_t* rows, int32_t* place,
                   int32_t* offsets, cudaStream_t st) {
  const size_t smem = plan_shared(E);
  // More than 48 KB, with the kernel's own variables (some hundred bytes), has
  // to be allowed.  Always the most: the limit is the kernel's, not the call's,
  // and another host thread may be about to launch a plan of more experts.
  if (smem > 47 * 1024) {
    const cudaError_t e = cudaFuncSetAttribute(k_moe_plan<Id>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               (int)plan_shared(EBC_MAX_EXPERTS));
    if (e != cudaSuccess) return e;
  }
  // CTAs of the cluster: a round of 1024 slots a CTA takes about a microsecond,
  // a larger cluster about as long to come together (1024 slots: 4.3 us with
  // one CTA, 4.8 with 8; 8192: 11.3, 5.3, and 5.8 with 16; 65,536: 71, 12.5, 9.1)
  unsigned C = n <= 1024 ? 1 : n <= 8192 ? 8 : 16;
  if (C > 8) {
    cudaError_t e = cudaFuncSetAttribute(k_moe_plan<Id>, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e == cudaSuccess && *v.plan_cluster == 0) e = ask_cluster<Id>(v.plan_cluster);
    if (e != cudaSuccess) return e;
    C = *v.plan_cluster;
  }
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
    const int64_t piece = 32 * scatter_vectors<V>() * (V / (int)sizeof(T));
    return launch_named(v, "k_moe_dispatch", st, k_moe_dispatch<T, V>,
                        dim3(row_grid(tokens * ((width + piece - 1) / piece), v.nsm)), dim3(32 * kRowWarps), 0, 1,
                        (const T*)d_x, ld_x, tokens, top, width, d_place, d_offsets, n_experts, (T*)d_xs, v.glob);
  }));
}

int ebc_moe_dispatch_mx(ebc_ctx* ctx, const uint8_t* d_codes, int64_t code_bytes, const uint8_t* d_scales,
                        int64_t scale_bytes, int64_t tokens, int top, const int32_t* d_place,
                        const int32_t* d_offsets, int n_experts, uint8_t* d_xs_codes, uint8_t* d_xs_scales,
                        void* stream) {
  constexpr int64_t kMost = (int64_t)1 << 24;   // a row of 2^24 values of 8 bits, and more than its scales
  if (!ctx || !routed_ok(tokens, top, n_experts) || code_bytes < 16 || code_bytes > kMost || code_bytes % 16 != 0 ||
      scale_bytes < 16 || scale_bytes > kMost || scale_bytes % 16 != 0 || !d_offsets || !aligned(d_offsets, 4))
    return EBC_ERR_INVALID_ARG;
  if (tokens > 0 && (!d_codes || !aligned(d_codes, 16) || !d_scales || !aligned(d_scales, 16) || !d_place ||
                     !aligned(d_place, 4) || !d_xs_codes || !aligned(d_xs_codes, 16) || !d_xs_scales ||
                     !aligned(d_xs_scales, 16)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || tokens == 0) return rc;
  const int64_t piece = 32 * scatter_vectors<16>(), vecs = (code_bytes + scale_bytes) / 16;
  return cuda_code(launch_named(v, "k_moe_dispatch_mx", st, k_moe_dispatch_mx,
                                dim3(row_grid(tokens * ((vecs + piece - 1) / piece), v.nsm)), dim3(32 * kRowWarps), 0,
                                1, (const uint4*)d_codes, code_bytes / 16, (const uint4*)d_scales, scale_bytes / 16,
                                tokens, top, d_place, d_offsets, n_experts, (uint4*)d_xs_codes, (uint4*)d_xs_scales,
                                v.glob));
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
    const int64_t piece = 32 * (V / (int)sizeof(T)) * gather_vectors<T, V>();
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
    // warps a slot: until there are 32 a SM, or until a warp's share is one round
    const int64_t n = tokens * top, round = 32 * (V / (int)sizeof(T)) * (V / (int)sizeof(T) >= 4 ? 4 : 8);
    int split = 1;
    while (split < kRowWarps && n * split < 32 * (int64_t)v.nsm && split * round < width) split *= 2;
    return launch_named(v, "k_moe_combine_grad", st, k_moe_combine_grad<T, V>, dim3(row_grid(n * split, v.nsm)),
                        dim3(32 * kRowWarps), 0, 1, (const T*)d_dy, ld_dy, (const T*)d_ys, ld_ys, tokens, top, width,
                        d_place, d_offsets, n_experts, d_weights, (T*)d_dys, d_dweights, split, v.glob);
  }));
}

}  // extern "C"
