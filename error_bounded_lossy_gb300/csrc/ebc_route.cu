// ebc_route.cu -- the router: each token's experts and weights from its scores,
// and the scores' gradient.  See include/ebc.h for the definitions.
#include <math_constants.h>

#include "ebc_types.cuh"

using namespace ebc;

namespace {

constexpr unsigned kAll = 0xffffffffu;
constexpr float kUlp = 1.1920929e-7f;   // 2^-23
constexpr int kGradWarps = 4;

// Values of 32 bits that order as floats do.  0 is what may not be chosen; a NaN
// is above everything; the two zeros are one value.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v + 0.f);
  return v != v ? ~0u : b & 0x80000000u ? ~b : b | 0x80000000u;
}
__device__ __forceinline__ float value_of(uint32_t k) {
  return k == ~0u ? CUDART_NAN_F : __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <typename R>
__device__ __forceinline__ R warp_sum(R v) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kAll, v, off);
  return v;
}
__device__ __forceinline__ float warp_max(float v) {   // (a NaN is ignored)
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kAll, v, off));
  return v;
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
  float scale;
  bool sigmoid, renorm, sums;   // sums: a group's score is the sum of two
};

// A warp's memory.
template <int N>
struct Room {
  float l[32 * N];
  float c[32 * N + 32];    // the choice's scores; a group starts at an odd distance from the next
  double d[32 * N];
  uint32_t key[34];        // the best, and one more
  int id[34];
};

// The choice in 64 bits, for tokens where 32 cannot tell two values apart: the
// same steps, written to be short.  Scores are computed again where c is in
// [lo, hi]; elsewhere what 32 bits say is enough.  Leaves the ids in room.id.
template <int N>
__device__ __noinline__ void choose_exactly(const RouteArgs& a, Room<N>& room, int pad, float most, double lo,
                                            double hi, int lane) {
  const int size = a.E / a.groups;
  double total = 1.0;
  if (!a.sigmoid) {
    total = 0.0;
    for (int e = lane; e < a.E; e += 32) total += exp((double)room.l[e] - (double)most);
    total = warp_sum(total);
  }
  for (int e = lane; e < a.E; e += 32) {
    const float l = room.l[e], b = a.bias ? a.bias[e] : 0.f;
    double c = (double)room.c[e + e / size * pad];
    if (l == -CUDART_INF_F || b == -CUDART_INF_F)
      c = -CUDART_INF;
    else if (c >= lo && c <= hi)
      c = (a.sigmoid ? 1.0 / (1.0 + exp(-(double)l)) : exp((double)l - (double)most) / total) + (double)b;
    room.d[e] = c;
  }
  __syncwarp();
  // a is better than b: larger, or a NaN
  auto better = [](double a, double b) { return a > b || (a != a && b == b); };
  unsigned kept = kAll;
  if (a.groups > 1) {
    double score = -CUDART_INF;
    if (lane < a.groups) {
      double first = -CUDART_INF, second = -CUDART_INF;
      for (int i = 0; i < size; ++i) {
        const double c = room.d[lane * size + i];
        if (better(c, first)) {
          second = first;
          first = c;
        } else if (better(c, second)) {
          second = c;
        }
      }
      score = a.sums && second != -CUDART_INF ? first + second : first;
    }
    int rank = 0;
    for (int g = 0; g < a.groups; ++g) {
      const double s = __shfl_sync(kAll, score, g);
      rank += better(s, score) || (!better(score, s) && g < lane);
    }
    kept = __ballot_sync(kAll, lane < a.groups && rank < a.keep);
  }
  for (int r = 0; r < a.top; ++r) {
    double best = -CUDART_INF;
    int at = INT32_MAX;
    for (int e = lane; e < a.E; e += 32) {
      if (a.groups > 1 && !(kept >> (e / size) & 1)) continue;
      // without a bias it is the logits that are compared
      const double c = room.d[e], v = c == -CUDART_INF || a.bias ? c : (double)room.l[e];
      if (better(v, best)) {
        best = v;
        at = e;
      }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) {
      const double v = __shfl_xor_sync(kAll, best, off);
      const int o = __shfl_xor_sync(kAll, at, off);
      if (better(v, best) || (!better(best, v) && o < at)) {
        best = v;
        at = o;
      }
    }
    if (lane == 0) {
      room.id[r] = at == INT32_MAX ? -1 : at;
      if (at != INT32_MAX) room.d[at] = -CUDART_INF;
    }
    __syncwarp();
  }
}

// A warp a token; lane i has the experts i * N to i * N + N - 1.
//
// The choice, in 32 bits: the (top + 1)-th largest of the lanes' largest values
// is a bound that at least top + 1 values reach; those that do (few more) are
// put into lanes by their order among the experts, and each counts how many
// come before it.  Where more than a warp of values reach it (ties), the best
// are taken one by one.
//
// Whether the choice is the one that the scores themselves give: the logits, as
// they are, order it where there is no bias; else a score in 32 bits is off by
// at most `err`, and where two values that decide are nearer than both may be
// off, the token is done again in 64 bits.
template <typename T, int N, int kWarps>
__global__ void __launch_bounds__(32 * kWarps) k_moe_route(RouteArgs a) {
  __shared__ Room<N> rooms[kWarps];
  pdl_enter();
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  Room<N>& room = rooms[w];
  const int size = a.E / a.groups, pad = a.groups > 1 && size % 2 == 0;
  const uint32_t inverse = ((1u << 20) + size - 1) / size;   // e / size is e * inverse >> 20 for e < 1024
  const bool scored = a.bias || (a.sums && a.groups > 1);
  float bias[N];
  uint32_t allowed = 0;   // a bit a value: an expert, not ruled out by its bias
  float bias_most = 0.f;
#pragma unroll
  for (int j = 0; j < N; ++j) {
    const int e = lane * N + j;
    bias[j] = a.bias && e < a.E ? a.bias[e] : 0.f;
    if (e < a.E && bias[j] != -CUDART_INF_F) allowed |= 1u << j;
    if (fabsf(bias[j]) < CUDART_INF_F) bias_most = fmaxf(bias_most, fabsf(bias[j]));
  }
  bias_most = warp_max(bias_most);
  for (int64_t t = (int64_t)blockIdx.x * kWarps + w; t < a.tokens; t += (int64_t)gridDim.x * kWarps) {
    const T* row = (const T*)a.logits + t * a.ld;
    float l[N], c[N];
    uint32_t alive = allowed;
    float most = -CUDART_INF_F;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = lane * N + j;
      l[j] = e < a.E ? to_f32(row[e]) : -CUDART_INF_F;
      if (l[j] == -CUDART_INF_F) alive &= ~(1u << j);
      most = fmaxf(most, l[j]);
    }
    float total = 1.f;
    if (!a.sigmoid && (scored || !a.renorm)) {
      most = shift_of(warp_max(most));
      total = 0.f;
#pragma unroll
      for (int j = 0; j < N; ++j) {
        c[j] = expf(l[j] - most);   // (of -infinity: 0)
        total += c[j];
      }
      total = warp_sum(total);
    }
    // How far a value in 32 bits may be off, with a margin.  Of the largest score
    // (1, or the softmax's 1 / total): for the sigmoid exp, the sum and the quotient
    // lose less than 2^-21; for the softmax the exponent's difference 2^-25 (it
    // grows as the score falls), exp and the quotient 2^-21, and the total's N + 5
    // roundings.  And the rounding of the bias's addition.
    const float err = a.sigmoid ? (9.f + bias_most) * kUlp : ((float)(N + 17) / total + bias_most) * kUlp;
    if (scored) {
#pragma unroll
      for (int j = 0; j < N; ++j) {
        const float s = a.sigmoid ? __fdividef(1.f, 1.f + expf(-l[j])) : __fdividef(c[j], total);
        c[j] = s + bias[j];
      }
    }
    __syncwarp();   // the room is free
#pragma unroll
    for (int j = 0; j < N; ++j) {
      const int e = lane * N + j;
      if (e < a.E) {
        room.l[e] = l[j];
        if (scored || a.groups > 1)
          room.c[e + (int)((uint32_t)e * inverse >> 20) * pad] =
              !(alive >> j & 1) ? -CUDART_INF_F : scored ? c[j] : l[j];
      }
    }
    __syncwarp();
    bool close = false;
    double lo = CUDART_INF, hi = -CUDART_INF;   // of the values that are too close
    if (a.groups > 1) {
      // `lanes` lanes a group, each its best two of every lanes-th value
      const int lanes_log2 = 31 - __clz(32 / a.groups), lanes = 1 << lanes_log2, g = lane >> lanes_log2;
      uint32_t first = 0, second = 0;
      if (g < a.groups)
        for (int i = lane & (lanes - 1); i < size; i += lanes) {
          const float v = room.c[g * (size + pad) + i];
          const uint32_t k = v == -CUDART_INF_F ? 0u : ordered(v);
          second = max(second, min(first, k));
          first = max(first, k);
        }
      for (int off = 1; off < lanes; off <<= 1) {
        const uint32_t f = __shfl_xor_sync(kAll, first, off), s = __shfl_xor_sync(kAll, second, off);
        second = max(max(second, s), min(first, f));
        first = max(first, f);
      }
      const uint32_t score = a.sums && second ? ordered(value_of(first) + value_of(second)) : first;
      int rank = 0;
      for (int i = 0; i < a.groups; ++i) {
        const uint32_t s = __shfl_sync(kAll, score, i << lanes_log2);
        rank += s > score || (s == score && i < g);
      }
      const bool one = g < a.groups && (lane & (lanes - 1)) == 0;   // (a group's first lane speaks for it)
      const unsigned kept = __ballot_sync(kAll, one && rank < a.keep);
      if (scored && a.keep < a.groups) {
        const unsigned in = __ballot_sync(kAll, one && rank == a.keep - 1), out = __ballot_sync(kAll, one && rank == a.keep);
        const uint32_t ki = __shfl_sync(kAll, score, __ffs(in) - 1), ko = __shfl_sync(kAll, score, __ffs(out) - 1);
        const float vi = value_of(ki), vo = value_of(ko);
        if (ki && ko && vi - vo <= 6.f * err) {   // (two values and a rounding each)
          close = true;
          lo = -CUDART_INF;
          hi = CUDART_INF;
        }
      }
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (!(kept >> (((uint32_t)(lane * N + j) * inverse >> 20) << lanes_log2 & 31) & 1)) alive &= ~(1u << j);
    }
    // the best top + 1
    uint32_t key[N], mine = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
      key[j] = alive >> j & 1 ? ordered(a.bias ? c[j] : l[j]) : 0u;
      mine = max(mine, key[j]);
    }
    uint32_t bound = 1, left = mine;
    for (int r = 0; r <= a.top; ++r) {
      const uint32_t m = __reduce_max_sync(kAll, left);
      bound = m ? m : 1u;
      if (!m) break;
      if (left == m) left = 0;
    }
    uint32_t reach = 0;
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (key[j] >= bound) reach |= 1u << j;
    int before = __popc(reach);
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const int v = __shfl_up_sync(kAll, before, off);
      if (lane >= off) before += v;
    }
    const int found = __shfl_sync(kAll, before, 31);
    before -= __popc(reach);
    // room.key and room.id: the best, the best first; zero and -1 behind them
    if (found <= 32) {
#pragma unroll
      for (int j = 0; j < N; ++j)
        if (reach >> j & 1) {
          room.key[before] = key[j];
          room.id[before] = lane * N + j;
          ++before;
        }
      __syncwarp();
      const uint32_t k = lane < found ? room.key[lane] : 0u;
      const int e = lane < found ? room.id[lane] : -1;
      int rank = 0;
      for (int i = 0; i < found; ++i) {
        const uint32_t o = __shfl_sync(kAll, k, i);
        rank += o > k || (o == k && i < lane);
      }
      if (lane >= found) rank = lane;
      __syncwarp();
      room.key[rank] = k;
      room.id[rank] = e;
      if (lane < 2) room.key[32 + lane] = 0u;
    } else {
      for (int r = 0; r <= a.top; ++r) {
        uint32_t best = 0;
        int at = 0;
#pragma unroll
        for (int j = 0; j < N; ++j)
          if (key[j] > best) {
            best = key[j];
            at = j;
          }
        const uint32_t m = __reduce_max_sync(kAll, best);
        const unsigned who = __ballot_sync(kAll, best == m);
        if (lane == __ffs(who) - 1) {
          room.key[r] = m;
          room.id[r] = m ? lane * N + at : -1;
#pragma unroll
          for (int j = 0; j < N; ++j)
            if (j == at) key[j] = 0;
        }
      }
    }
    __syncwarp();
    if (a.bias) {
      const uint32_t k = lane < a.top ? room.key[lane] : 0u, o = lane < a.top ? room.key[lane + 1] : 0u;
      const float v = value_of(k), u = value_of(o);
      const bool near = k && o && v - u <= 2.f * err;
      if (__any_sync(kAll, near)) {
        close = true;
        // whatever is within reach of a pair (and of a run of them) is computed again
        double from = near ? (double)u - 4.0 * err : CUDART_INF, to = near ? (double)v + 4.0 * err : -CUDART_INF;
#pragma unroll
        for (int off = 16; off > 0; off >>= 1) {
          from = fmin(from, __shfl_xor_sync(kAll, from, off));
          to = fmax(to, __shfl_xor_sync(kAll, to, off));
        }
        lo = fmin(lo, from);
        hi = fmax(hi, to);
      }
    }
    if (close) {
      choose_exactly<N>(a, room, pad, most, lo, hi, lane);
      __syncwarp();
    }
    // weights, a lane a choice
    const int id = lane < a.top ? room.id[lane] : -1;
    const float x = id >= 0 ? room.l[id] : -CUDART_INF_F;
    float s;
    if (a.renorm) {
      // shifted by the largest chosen, so that no sum is zero: for the sigmoid
      // only below 0, exp(x - m) / (1 + exp(x)) with m = 0 from there on
      const float m = shift_of(warp_max(x));
      if (a.sigmoid)
        s = x <= 0.f ? expf(x - fminf(m, 0.f)) / (1.f + expf(x)) : 1.f / (1.f + expf(-x));
      else
        s = expf(x - m);
      if (id < 0) s = 0.f;
      const float sum = warp_sum(s);
      // (a softmax with a NaN or +infinity in its row is NaN, whatever was chosen)
      s = id < 0 ? 0.f : total == total ? s / sum : total;
    } else {
      s = id < 0 ? 0.f : a.sigmoid ? 1.f / (1.f + expf(-x)) : expf(x - most) / total;
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
cudaError_t route_n(const CallView& v, const RouteArgs& a, cudaStream_t st) {
  constexpr int kWarps = N == 32 ? 2 : 4;
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
  const RouteArgs a{d_logits, d_bias, d_ids, d_weights, ld_logits, tokens, n_experts, top,
                    keep_groups == groups ? 1 : groups, keep_groups == groups ? 1 : keep_groups, scale,
                    score == EBC_SIGMOID, renormalize != 0, group_top == 2};
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
