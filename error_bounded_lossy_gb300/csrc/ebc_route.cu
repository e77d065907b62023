// ebc_route.cu -- the router: each token's experts and weights from its scores,
// and the scores' gradient.  See include/ebc.h for the definitions.
#include <math_constants.h>

#include "ebc_mx8.cuh"

using namespace ebc;

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kUlp = 1.1920929e-7f;   // 2^-23
constexpr int kGradWarps = 4;

template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {   // (a NaN is ignored)
  float r;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
  return r;
}
__device__ __forceinline__ float max_or_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// What the largest exponent is taken from: nothing where there is none.
__device__ __forceinline__ float shift_of(float most) { return most == -CUDART_INF_F ? 0.f : most; }

struct RouteArgs {
  const void* logits;
  const float* bias;
  int32_t* ids;
  float* weights;
  int64_t ld, tokens;
  int E, top, groups, keep;
  uint32_t inverse;             // e / (E / groups) is e * inverse >> 20 for e < 1024
  int group_lanes_log2;         // lanes of a group, where a group is whole lanes and a power of two of them; else -1
  float scale;
  bool sigmoid, renorm, sums;   // sums: a group's score is the sum of two
  bool wide, wide_bias;         // a lane's logits, and biases, are whole vectors
};

// A warp's memory.  Values: a group starts at an odd distance from the next.
template <int N>
struct Room {
  union {
    float c[32 * N + 32];
    int64_t k[32 * N];
  };
  // the candidates (a value and its expert each), then the best of them in their
  // order, and one that nobody reads
  float2 slot[36];
  __device__ __forceinline__ float value(int i) const { return slot[i].x; }
  __device__ __forceinline__ int id(int i) const { return __float_as_int(slot[i].y); }
  __device__ __forceinline__ void put(int i, float v, int e) { slot[i] = make_float2(v, __int_as_float(e)); }
  static constexpr int kNowhere = 35;
};

// ---- scores in 64 bits, for values that 32 cannot tell apart ----
// The sum of a softmax's exponentials.
template <typename T>
__device__ __noinline__ double exact_total(const T* row, int E, float most, int lane) {
  double sum = 0.0, last = 0.0;
  float l_last = CUDART_NAN_F;   // (like nothing)
  for (int e = lane; e < E; e += 32) {
    const float l = to_f32(row[e]);
    if (l != l_last) last = exp((double)l - (double)most);
    l_last = l;
    sum += last;
  }
  return warp_sum(sum);
}
// The choice's value of an expert.
template <typename T>
__device__ __noinline__ double exact_value(const RouteArgs& a, const T* row, int e, float most, double total) {
  const double l = (double)to_f32(row[e]);
  return (a.sigmoid ? 1.0 / (1.0 + exp(-l)) : exp(l - (double)most) / total) + (a.bias ? (double)a.bias[e] : 0.0);
}

// Numbers in their order as integers, NaN the largest: this chip has few units for
// 64-bit floating point, and its comparisons are of them (8192 x 256 with a bias 11.6
// -> 11.0 us, rows of equal scores 277 -> 49).
__device__ __forceinline__ int64_t key_of(double v) {
  const int64_t bits = __double_as_longlong(v), low = 0x7fffffffffffffffll;
  if ((bits & low) == 0) return 0;   // (both zeros)
  return (bits & low) > 0x7ff0000000000000ll ? low : bits ^ ((bits >> 63) & low);
}
__device__ __forceinline__ int64_t key_of(float v) {
  const int32_t bits = __float_as_int(v), low = 0x7fffffff;
  if ((bits & low) == 0) return 0;
  return (bits & low) > 0x7f800000 ? low : bits ^ ((bits >> 31) & low);
}
__device__ __forceinline__ double of_key(int64_t k) { return __longlong_as_double(k ^ ((k >> 63) & 0x7fffffffffffffffll)); }
constexpr int64_t kNone = -0x7ff0000000000001ll;   // of -infinity: below any other

// The whole choice in 64 bits, for rows with a NaN and for ties of more values
// than a warp has lanes: the same steps, written to be short.  A NaN is above
// everything.  Leaves the ids in the slots.
template <typename T, int N>
__device__ __noinline__ void choose_exactly(const RouteArgs& a, Room<N>& room, const T* row, float most, bool scored,
                                            int lane) {
  const int size = a.E / a.groups;
  const double total = scored && !a.sigmoid ? exact_total(row, a.E, most, lane) : 1.0;
  __syncwarp();
  // (a value like the lane's one before is not computed again: most where rows tie)
  float l_last = 0.f, b_last = 0.f;
  int64_t last = kNone;
  bool any = false;
  for (int e = lane; e < a.E; e += 32) {
    const float l = to_f32(row[e]), b = a.bias ? a.bias[e] : 0.f;
    if (scored && !(any && l == l_last && b == b_last)) {
      last = key_of(exact_value(a, row, e, most, total));
      l_last = l;
      b_last = b;
      any = true;
    }
    room.k[e] = l == -CUDART_INF_F || b == -CUDART_INF_F ? kNone : scored ? last : key_of(l);
  }
  __syncwarp();
  unsigned kept = kAll;
  if (a.groups > 1) {
    int64_t score = kNone;
    if (lane < a.groups) {
      int64_t first = kNone, second = kNone;
      for (int i = 0; i < size; ++i) {
        const int64_t c = room.k[lane * size + i];
        second = c > first ? first : c > second ? c : second;
        first = c > first ? c : first;
      }
      score = a.sums && second != kNone ? key_of(of_key(first) + of_key(second)) : first;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const int64_t s = __shfl_sync(kAll, score, g);
      rank += s > score || (s == score && g < lane);
    }
    kept = __ballot_sync(kAll, lane < a.groups && rank < a.keep);
    for (int e = lane; e < a.E; e += 32)
      if (!(kept >> (e / size) & 1))
        room.k[e] = kNone;
      else if (scored && !a.bias && room.k[e] != kNone)   // without a bias it is the logits that are compared
        room.k[e] = key_of(to_f32(row[e]));
    __syncwarp();
  }
  for (int r = 0; r < a.top; ++r) {
    int64_t best = kNone;
    int at = INT32_MAX;
    for (int e = lane; e < a.E; e += 32)
      if (room.k[e] > best) {
        best = room.k[e];
        at = e;
      }
#pragma unroll 1
    for (int off = 16; off > 0; off >>= 1) {
      const int64_t v = __shfl_xor_sync(kAll, best, off);
      const int o = __shfl_xor_sync(kAll, at, off);
      if (v > best || (v == best && o < at)) {
        best = v;
        at = o;
      }
    }
    if (lane == 0) {
      room.put(r, 0.f, at == INT32_MAX ? -1 : at);
      if (at != INT32_MAX) room.k[at] = kNone;
    }
    __syncwarp();
  }
}

// A lane's N values from lane * N on (of E), `missing` past the end.
template <typename T, int N>
__device__ __forceinline__ void load_lane(const T* p, int E, int lane, bool wide, float missing, float (&v)[N]) {
  if (wide) {
    constexpr int kV = N < 8 ? N : 8;
    Values<T, kV> r[N / kV];
#pragma unroll
    for (int i = 0; i < N / kV; ++i)
      if (lane * N < E) r[i].load(p + lane * N + i * kV);
#pragma unroll
    for (int i = 0; i < N / kV; ++i) {
      float f[kV];
      r[i].get(f);
#pragma unroll
      for (int j = 0; j < kV; ++j) v[i * kV + j] = lane * N < E ? f[j] : missing;
    }
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j) v[j] = lane * N + j < E ? to_f32(p[lane * N + j]) : missing;
  }
}

// Puts the experts of the set bits (bit j of a lane: expert lane * N + j) into the
// slots in their order, with their values; returns how many, and writes nothing
// where they are more than a warp.
template <int N>
__device__ __forceinline__ int gather(Room<N>& room, uint32_t bits, const float (&v)[N], int lane) {
  const int mine = __popc(bits);
  int at = mine;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int o = __shfl_up_sync(kAll, at, off);
    if (lane >= off) at += o;
  }
  const int all = __shfl_sync(kAll, at, 31);
  at -= mine;
  __syncwarp();
  if (all <= 32) {
    // (a store for each value, not a branch: most of them nowhere)
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const bool set = bits >> j & 1;
      room.put(set ? at : Room<N>::kNowhere, v[j], lane * N + j);
      at += set;
    }
  }
  __syncwarp();
  return all;
}

// The groups' ranks from sums in 64 bits of the `near` ones' largest values, which
// are among the `found` of room.id, and from the others' as they are (score: half of
// a sum).
template <typename T, int N>
__device__ __noinline__ int settle_groups(const RouteArgs& a, Room<N>& room, const T* row, float most, int found,
                                          bool near, float score, int log2, int lane) {
  const double total = a.sigmoid ? 1.0 : exact_total(row, a.E, most, lane);
  const int e = lane < found ? room.id(lane) : 0, g = lane >> log2;
  const int64_t value = key_of(exact_value(a, row, e, most, total));
  const int eg = (int)((uint32_t)e * a.inverse >> 20);
  int64_t first = kNone, second = kNone;
#pragma unroll 1
  for (int i = 0; i < found; ++i) {
    const int64_t v = __shfl_sync(kAll, value, i);
    if (__shfl_sync(kAll, eg, i) == g) {
      second = v > first ? first : v > second ? v : second;
      first = v > first ? v : first;
    }
  }
  const int64_t sure = !near ? key_of(a.sums ? 2. * (double)score : (double)score)
                       : a.sums && second > kNone ? key_of(of_key(first) + of_key(second)) : first;
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < a.groups; ++i) {
    const int64_t o = __shfl_sync(kAll, sure, i << log2);
    rank += o > sure || (o == sure && i < g);
  }
  return rank;
}

// The order of the `found` best in room.id by their values in 64 bits.
template <typename T, int N>
__device__ __noinline__ void settle_order(const RouteArgs& a, Room<N>& room, const T* row, float most, int found,
                                          int lane) {
  const double total = a.sigmoid ? 1.0 : exact_total(row, a.E, most, lane);
  const int e = lane < found ? room.id(lane) : -1;
  const int64_t value = e >= 0 ? key_of(exact_value(a, row, e, most, total)) : kNone;
  int rank = 0;
#pragma unroll 1
  for (int i = 0; i < found; ++i) {
    const int64_t u = __shfl_sync(kAll, value, i);
    const int n = __shfl_sync(kAll, e, i);
    rank += u > value || (u == value && n < e);
  }
  __syncwarp();
  if (lane < found) room.put(rank, 0.f, e);
  __syncwarp();
}

// A warp a token; lane i has the experts i * N to i * N + N - 1, whose values in
// 32 bits are -infinity where they may not be chosen.
//
// The choice: the top-th largest of the lanes' largest values is a bound that at
// least `top` values reach; those that do (few more) are put into lanes in the
// experts' order, and each counts the ones before it.
//
// Whether that is the choice that the scores themselves give: the logits order
// it, as they are, where there is no bias; else a value in 32 bits is off by at
// most `err`, and where two that decide are nearer than both may be off, those
// few are computed again in 64 bits, a lane each, and compared so (two equal
// logits with equal biases are equal, and need none of it).  The same for the
// groups at the border of the kept ones.  With 256 experts that is one token in
// some hundreds, and 2 to 3 us of a batch of 8192 (a token's few values in 64 bits
// a lane each; its whole row so took 30).
//
// Bound by issue: some 600 instructions a token, 300 more for the scores of a
// bias, 350 more for groups.  8192 tokens x 256 experts, 8 chosen: 7.2 us by the
// logits, 11.0 with a bias, 13.7 with both; x 64: 5.7.  A search a choice took 15.8,
// 46 and 58.  A token alone takes 2.5 to 4 us of latency.  The registers of eight CTAs an
// SM are 64, in which 65 to 256 experts spill 20 to 96 bytes; 257 to 512 have 128 (fp32
// spills 36), more have 196 to 229 and eight warps an SM (8192 x 1024: 18.3, 34 and 41 us).
// A finite mask in the bias (-1e9) makes `err` so large that every token goes to
// choose_exactly: 118 us of 8192 x 256.
template <typename T, int N, int kWarps>
__global__ void __launch_bounds__(32 * kWarps, N <= 8 ? 8 : 4) k_moe_route(const __grid_constant__ RouteArgs a) {
  __shared__ Room<N> rooms[kWarps];
  pdl_enter();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Room<N>& room = rooms[w];
  const bool scored = a.bias || (a.sums && a.groups > 1);
  float bias_most = -1.f;   // (not known yet)
  for (int64_t t = (int64_t)blockIdx.x * kWarps + w; t < a.tokens; t += (int64_t)gridDim.x * kWarps) {
    const T* row = (const T*)a.logits + t * a.ld;
    float c[N], b[N];   // c: first the logits
    load_lane<T, N>(row, a.E, lane, a.wide, -CUDART_INF_F, c);
    if (a.bias) {
      load_lane<float, N>(a.bias, a.E, lane, a.wide_bias, 0.f, b);
      if (bias_most < 0.f) {
        bias_most = 0.f;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (fabsf(b[j]) < CUDART_INF_F) bias_most = fmaxf(bias_most, fabsf(b[j]));
        bias_most = warp_max(bias_most);
      }
    } else {
      bias_most = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) b[j] = 0.f;
    }
    float most = 0.f, total = 1.f;
    if (!a.sigmoid && (scored || !a.renorm)) {
      most = c[0];
#pragma unroll
      for (int j = 1; j < N; ++j) most = fmaxf(most, c[j]);
      most = shift_of(warp_max(most));
      total = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) total += __expf(c[j] - most);   // (of -infinity: 0)
      total = warp_sum(total);
    }
    // How far a value in 32 bits may be off, with a margin.  Of the largest score
    // (1, or the softmax's 1 / total): for the sigmoid the exponential, which is off
    // by 2 + 1.2 |l| units of which s (1 - s) counts, the sum and the quotient lose
    // less than 2^-21; for the softmax the exponential and the quotient 2^-21 (more
    // where the score is smaller by more), and the total's N + 5 roundings and its
    // terms' errors 2^-19.  And the rounding of the bias's addition.
    const float err = a.sigmoid ? (9.f + bias_most) * kUlp : ((float)(N + 48) / total + bias_most) * kUlp;
    if (scored) {
      const float part = __fdividef(1.f, total);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float s = a.sigmoid ? __fdividef(1.f, 1.f + __expf(-c[j])) : __expf(c[j] - most) * part;
        c[j] = c[j] == -CUDART_INF_F ? c[j] : s + b[j];
      }
    }
    float top1 = c[0];
#pragma unroll
    for (int j = 1; j < N; ++j) top1 = max_or_nan(top1, c[j]);
    bool generic = __any_sync(kAll, top1 != top1);   // a NaN
    if (a.groups > 1 && !generic) {
      // a group's largest two, in each of its lanes
      float first = -CUDART_INF_F, second = -CUDART_INF_F;
      int log2 = a.group_lanes_log2;
      if (log2 >= 0) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          second = fmaxf(second, fminf(first, c[j]));
          first = fmaxf(first, c[j]);
        }
      } else {
        const int size = a.E / a.groups, pad = size % 2 == 0;
        __syncwarp();
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const int e = lane * N + j;
          if (e < a.E) room.c[e + (int)((uint32_t)e * a.inverse >> 20) * pad] = c[j];
        }
        __syncwarp();
        log2 = 31 - __clz(32 / a.groups);
        if (lane >> log2 < a.groups)
          for (int i = lane & ((1 << log2) - 1); i < size; i += 1 << log2) {
            const float v = room.c[(lane >> log2) * (size + pad) + i];
            second = fmaxf(second, fminf(first, v));
            first = fmaxf(first, v);
          }
      }
      const int g = lane >> log2;
#pragma unroll 1
      for (int off = 1; off < 1 << log2; off <<= 1) {
        const float f = __shfl_xor_sync(kAll, first, off), s = __shfl_xor_sync(kAll, second, off);
        second = fmaxf(fmaxf(second, s), fminf(first, f));
        first = fmaxf(first, f);
      }
      // (half of the sum, which is exact but for numbers far below any `err`: two finite
      // values may add up to more than fp32 holds)
      const float score = !a.sums ? first : second > -CUDART_INF_F ? .5f * first + .5f * second : .5f * first;
      int rank = 0;
      for (int i = 0; i < a.groups; ++i) {
        const float s = __shfl_sync(kAll, score, i << log2);
        rank += s > score || (s == score && i < g);
      }
      const bool one = g < a.groups && (lane & ((1 << log2) - 1)) == 0;   // (a group's first lane speaks for it)
      if (scored && a.keep < a.groups) {
        const unsigned in = __ballot_sync(kAll, one && rank == a.keep - 1), out = __ballot_sync(kAll, one && rank == a.keep);
        const float vi = __shfl_sync(kAll, score, __ffs(in) - 1), vo = __shfl_sync(kAll, score, __ffs(out) - 1);
        const float reach = a.sums ? 3.f * err : 6.f * err;   // (two values and a rounding each, or half of them)
        if (vo > -CUDART_INF_F && vi - vo <= reach) {
          // what decides: the largest of the groups that are that near
          const bool near = score <= vi + reach && score >= vo - reach;
          const float from = near ? (a.sums && second > -CUDART_INF_F ? second : first) - 2.f * err : CUDART_INF_F;
          uint32_t bits = 0;
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const int eg = (int)((uint32_t)(lane * N + j) * a.inverse >> 20) & 31;
            const float least = __shfl_sync(kAll, from, eg << log2 & 31);
            if (c[j] >= least && c[j] > -CUDART_INF_F) bits |= 1u << j;
          }
          const int found = gather(room, bits, c, lane);
          generic = found > 32;
          if (!generic) rank = settle_groups<T, N>(a, room, row, most, found, near, score, log2, lane);
        }
      }
      const unsigned kept = __ballot_sync(kAll, one && rank < a.keep);
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const uint32_t eg = a.group_lanes_log2 >= 0 ? (uint32_t)g : (uint32_t)(lane * N + j) * a.inverse >> 20;
        if (!(kept >> (eg << log2 & 31) & 1)) c[j] = -CUDART_INF_F;
      }
      if (scored && !a.bias) {   // the choice compares the logits
        float l[N];
        load_lane<T, N>(row, a.E, lane, a.wide, -CUDART_INF_F, l);
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (c[j] != -CUDART_INF_F) c[j] = l[j];
      }
      top1 = c[0];
#pragma unroll
      for (int j = 1; j < N; ++j) top1 = fmaxf(top1, c[j]);
    }
    int id = -1;
    if (!generic) {
      // at least the best `top`, and whatever may be among them
      auto from = [&](float bound) {
        if (a.bias) bound -= 2.f * err;
        uint32_t bits = 0;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (c[j] >= bound && c[j] > -CUDART_INF_F) bits |= 1u << j;
        return gather(room, bits, c, lane);
      };
      float bound = -CUDART_INF_F, left = top1;
#pragma unroll 1
      for (int r = 0; r < a.top; ++r) {
        bound = warp_max(left);
        if (bound == -CUDART_INF_F) break;
        if (left == bound) left = -CUDART_INF_F;
      }
      int found = from(bound);
      if (found > 32 && a.bias) {
        // many choices, or few lanes with what may be chosen: as many of the values
        // themselves, equal ones of a lane once (8 of two groups of 32: 369 -> 16 us of
        // 8192 tokens, 24 of 256: 818 -> 24, in choose_exactly as it then was)
        left = top1;
#pragma unroll 1
        for (int r = 0; r < a.top; ++r) {
          bound = warp_max(left);
          if (bound == -CUDART_INF_F) break;
          if (left == bound) {
            left = -CUDART_INF_F;
#pragma unroll
            for (int j = 0; j < N; ++j)
              if (c[j] < bound) left = fmaxf(left, c[j]);
          }
        }
        found = from(bound);
      }
      if (found <= 32) {
        float v = lane < found ? room.value(lane) : -CUDART_INF_F;
        int e = lane < found ? room.id(lane) : -1, rank = 0;
#pragma unroll 4
        for (int i = 0; i < found; ++i) {
          const float o = room.value(i);
          rank += o > v || (o == v && i < lane);
        }
        if (lane >= found) rank = lane;
        __syncwarp();
        room.put(rank, v, e);
        __syncwarp();
        if (a.bias) {
          // is each of the best far enough from the next, or the same as it
          v = room.value(lane);
          const float o = __shfl_down_sync(kAll, v, 1);
          bool near = lane < a.top && lane < 31 && o > -CUDART_INF_F && v - o <= 2.f * err;
          if (__any_sync(kAll, near)) {
            e = room.id(lane);
            const float x = e >= 0 ? to_f32(row[e]) : 0.f, b = e >= 0 ? a.bias[e] : 0.f;
            const float ox = __shfl_down_sync(kAll, x, 1), ob = __shfl_down_sync(kAll, b, 1);
            near = near && !(x == ox && b == ob);
            if (__any_sync(kAll, near)) settle_order<T, N>(a, room, row, most, found, lane);
          }
        }
        id = lane < a.top ? room.id(lane) : -1;
      } else if (!a.bias) {
        // ties of more than a warp of values: the best one by one
#pragma unroll 1
        for (int r = 0; r < a.top; ++r) {
          float best = c[0];
          int at = 0;
#pragma unroll
          for (int j = 1; j < N; ++j)
            if (c[j] > best) {
              best = c[j];
              at = j;
            }
          const float m = warp_max(best);
          if (m == -CUDART_INF_F) break;
          const int winner = __ffs(__ballot_sync(kAll, best == m)) - 1;
          const int e = __shfl_sync(kAll, lane * N + at, winner);
          if (lane == r) id = e;
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (lane == winner && j == at) c[j] = -CUDART_INF_F;
        }
      } else {
        generic = true;
      }
    }
    if (generic) {
      choose_exactly<T, N>(a, room, row, most, scored, lane);
      id = lane < a.top ? room.id(lane) : -1;
      __syncwarp();
    }
    // weights, a lane a choice
    const float x = id >= 0 ? to_f32(row[id]) : -CUDART_INF_F;
    float s = 0.f;
    if (a.renorm) {
      // shifted by the largest chosen, so that no sum is zero: for the sigmoid
      // only below 0, exp(x - m) / (1 + exp(x)) with m = 0 from there on
      float m = shift_of(warp_max(x));
      if (a.sigmoid) m = fminf(m, 0.f);
      const bool high = a.sigmoid && x > 0.f;
      s = expf(high ? -x : x - m);
      if (a.sigmoid) s = (high ? 1.f : s) / (1.f + (high ? s : expf(x)));
      if (id < 0) s = 0.f;
      const float sum = warp_sum(s);
      // (a softmax with a NaN or +infinity in its row is NaN, whatever was chosen)
      s = id < 0 ? 0.f : total == total ? s / sum : total;
    } else if (id >= 0) {
      s = expf(a.sigmoid ? -x : x - most);
      s = a.sigmoid ? 1.f / (1.f + s) : s / total;
    }
    if (lane < a.top) {
      a.ids[t * a.top + lane] = id;
      a.weights[t * a.top + lane] = a.scale * s;
    }
  }
}

struct RouteGradArgs {
  const float* dweights;
  const void* logits;
  const int32_t* ids;
  void* dlogits;
  Glob* glob;
  int64_t ld, tokens;
  int E, top;
  float scale;
  bool sigmoid, renorm;
};

// The gradient of a token's scores, a warp a token and a lane a choice.  With
// g = scale * dweights, u the chosen scores' shares (s / sum of s):
//   softmax, renormalised   dl = u (g - sum of u g)
//   sigmoid, renormalised   dl = u (g - sum of u g) (1 - s)
//   sigmoid                 dl = g s (1 - s)
//   softmax                 dl = p ([chosen] g - sum of p g), for every expert
// and zero for what was not chosen.  Bound by bandwidth: it writes a value for
// each score, and reads only the softmax's scores that are not renormalised.
template <typename T>
__global__ void __launch_bounds__(32 * kGradWarps) k_moe_route_grad(RouteGradArgs a) {
  __shared__ float rows[kGradWarps][EBC_MAX_EXPERTS];
  pdl_enter();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  float* out = rows[w];
  const bool dense = !a.sigmoid && !a.renorm;
  for (int64_t t = (int64_t)blockIdx.x * kGradWarps + w; t < a.tokens; t += (int64_t)gridDim.x * kGradWarps) {
    const T* row = (const T*)a.logits + t * a.ld;
    int id = lane < a.top ? a.ids[t * a.top + lane] : -1;
    if (id >= a.E) {
      record_error(a.glob, EBC_ERR_INVALID_ARG);
      id = -1;
    }
    const float x = id >= 0 ? to_f32(row[id]) : -CUDART_INF_F;
    const float g = id >= 0 ? a.scale * a.dweights[t * a.top + lane] : 0.f;
    float d = 0.f, most = 0.f, total = 1.f;
    if (dense) {
      most = -CUDART_INF_F;
      for (int e = lane; e < a.E; e += 32) most = fmaxf(most, to_f32(row[e]));
      most = shift_of(warp_max(most));
      total = 0.f;
      for (int e = lane; e < a.E; e += 32) total += expf(to_f32(row[e]) - most);
      total = warp_sum(total);
      if (id >= 0) d = expf(x - most) / total * g;
    } else if (a.renorm) {
      const float m = shift_of(warp_max(x));
      float s = 0.f;
      if (id >= 0)
        s = !a.sigmoid ? expf(x - m)
            : x <= 0.f ? expf(x - fminf(m, 0.f)) / (1.f + expf(x))
                       : 1.f / (1.f + expf(-x));
      const float sum = warp_sum(s);
      const float u = id >= 0 ? s / sum : 0.f;
      d = u * (g - warp_sum(u * g));
      if (a.sigmoid) d *= 1.f / (1.f + expf(x));
    } else if (id >= 0) {
      d = g * (1.f / (1.f + expf(-x))) * (1.f / (1.f + expf(x)));
    }
    if (id < 0) d = 0.f;
    __syncwarp();   // the row before has been written
    for (int e = lane; e < a.E; e += 32) out[e] = 0.f;
    __syncwarp();
    // (an id that is there twice: its parts one after the other)
    const unsigned same = __match_any_sync(kAll, id);
    if (__any_sync(kAll, id >= 0 && (same & (same - 1)))) {
      for (int r = 0; r < a.top; ++r) {
        if (lane == r && id >= 0) out[id] += d;
        __syncwarp();
      }
    } else if (id >= 0) {
      out[id] = d;
    }
    const float all = dense && total != 0.f ? warp_sum(d) / total : 0.f;   // (0: every expert is masked out)
    __syncwarp();
    T* dst = (T*)a.dlogits + t * a.E;
    for (int e = lane; e < a.E; e += 32) {
      float v = out[e];
      if (dense) v -= expf(to_f32(row[e]) - most) * all;
      dst[e] = from_f32<T>(v);
    }
  }
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

bool routed_ok(int type, int64_t tokens, int E, int top, int score, int64_t ld) {
  return type_bytes(type) && tokens >= 0 && E >= 1 && E <= EBC_MAX_EXPERTS && top >= 1 && top <= EBC_MAX_TOP &&
         tokens <= INT32_MAX / top && (score == EBC_SOFTMAX || score == EBC_SIGMOID) && ld >= E &&
         ld <= ((int64_t)1 << 40);
}

// CTAs for the tokens' warps, at most `turns` full turns of the machine.
unsigned grid(int64_t tokens, int warps, int nsm, int turns) {
  const int64_t want = (tokens + warps - 1) / warps, most = (int64_t)nsm * (64 / warps) * turns;
  return (unsigned)(want < most ? want : most);
}

template <typename T, int N>
cudaError_t route_n(const CallView& v, RouteArgs a, cudaStream_t st) {
  constexpr int kWarps = N == 32 ? 2 : 4, kBytes = (N < 8 ? N : 8) * (int)sizeof(T);
  a.wide = a.E % N == 0 && ((uintptr_t)a.logits | (uintptr_t)(a.ld * (int64_t)sizeof(T))) % kBytes == 0;
  a.wide_bias = a.E % N == 0 && (uintptr_t)a.bias % ((N < 8 ? N : 8) * 4) == 0;
  const int size = a.E / a.groups, lanes = size / N;
  a.group_lanes_log2 = -1;
  if (size % N == 0 && (lanes & (lanes - 1)) == 0)
    for (a.group_lanes_log2 = 0; 1 << a.group_lanes_log2 < lanes;) ++a.group_lanes_log2;
  return launch_named(v, "k_moe_route", st, k_moe_route<T, N, kWarps>, dim3(grid(a.tokens, kWarps, v.nsm, 1)),
                      dim3(32 * kWarps), 0, 1, a);
}

template <typename T>
cudaError_t route_t(const CallView& v, const RouteArgs& a, cudaStream_t st) {
  if (a.E <= 32) return route_n<T, 1>(v, a, st);
  if (a.E <= 64) return route_n<T, 2>(v, a, st);
  if (a.E <= 128) return route_n<T, 4>(v, a, st);
  if (a.E <= 256) return route_n<T, 8>(v, a, st);
  if (a.E <= 512) return route_n<T, 16>(v, a, st);
  return route_n<T, 32>(v, a, st);
}

}  // namespace

extern "C" {

int ebc_moe_route(ebc_ctx* ctx, const void* d_logits, int64_t ld_logits, int type, int64_t tokens, int n_experts,
                  int top, int score, const float* d_bias, int groups, int keep_groups, int group_top,
                  int renormalize, float scale, int32_t* d_ids, float* d_weights, void* stream) {
  if (!ctx || !routed_ok(type, tokens, n_experts, top, score, ld_logits) || groups < 1 || groups > EBC_MAX_GROUPS ||
      n_experts % groups != 0 || keep_groups < 1 || keep_groups > groups || group_top < 1 || group_top > 2 ||
      !(scale >= -3.4028235e38f && scale <= 3.4028235e38f) || !aligned(d_bias, 4))
    return EBC_ERR_INVALID_ARG;
  const int b = type_bytes(type);
  if (tokens > 0 && (!d_logits || !aligned(d_logits, b) || !d_ids || !aligned(d_ids, 4) || !d_weights ||
                     !aligned(d_weights, 4)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || tokens == 0) return rc;
  // (all groups kept: no group decides anything)
  RouteArgs a = {};
  a.logits = d_logits;
  a.bias = d_bias;
  a.ids = d_ids;
  a.weights = d_weights;
  a.ld = ld_logits;
  a.tokens = tokens;
  a.E = n_experts;
  a.top = top;
  a.groups = keep_groups == groups ? 1 : groups;
  a.keep = keep_groups == groups ? 1 : keep_groups;
  const uint32_t size = (uint32_t)(a.E / a.groups);
  a.inverse = ((1u << 20) + size - 1) / size;
  a.scale = scale;
  a.sigmoid = score == EBC_SIGMOID;
  a.renorm = renormalize != 0;
  a.sums = group_top == 2;
  if (type == EBC_F32) return cuda_code(route_t<float>(v, a, st));
  if (type == EBC_BF16) return cuda_code(route_t<__nv_bfloat16>(v, a, st));
  return cuda_code(route_t<__half>(v, a, st));
}

int ebc_moe_route_grad(ebc_ctx* ctx, const float* d_dweights, const void* d_logits, int64_t ld_logits, int type,
                       int64_t tokens, int n_experts, int top, const int32_t* d_ids, int score, int renormalize,
                       float scale, void* d_dlogits, void* stream) {
  if (!ctx || !routed_ok(type, tokens, n_experts, top, score, ld_logits) ||
      !(scale >= -3.4028235e38f && scale <= 3.4028235e38f))
    return EBC_ERR_INVALID_ARG;
  const int b = type_bytes(type);
  if (tokens > 0 && (!d_dweights || !aligned(d_dweights, 4) || !d_logits || !aligned(d_logits, b) || !d_ids ||
                     !aligned(d_ids, 4) || !d_dlogits || !aligned(d_dlogits, b)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || tokens == 0) return rc;
  const RouteGradArgs a{d_dweights, d_logits, d_ids, d_dlogits, v.glob, ld_logits, tokens, n_experts, top, scale,
                        score == EBC_SIGMOID, renormalize != 0};
  auto launch = [&](auto one) {
    return launch_named(v, "k_moe_route_grad", st, k_moe_route_grad<decltype(one)>,
                        dim3(grid(tokens, kGradWarps, v.nsm, 1)), dim3(32 * kGradWarps), 0, 1, a);
  };
  if (type == EBC_F32) return cuda_code(launch(float()));
  if (type == EBC_BF16) return cuda_code(launch(__nv_bfloat16()));
  return cuda_code(launch(__half()));
}

}  // extern "C"
