// ebc_types.cuh -- what the expert-parallel and 4-bit calls share: a context as
// they see it, element types, and row vectors (loads and stores of V bytes,
// converted from and to fp32).
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "ebc_internal.cuh"

namespace ebc {

// What the expert-parallel and 4-bit entry points need of a context: the
// device's SMs, the CTAs that a plan's cluster may have (0: not asked yet), the
// polls of a kernel's first wait (a test aid), the error word that the kernels
// record into, and the profiler.  begin_call checks the
// context, makes its device current for as long as the view lives, and notes
// the stream as that of the last call (defined with the C ABI).
struct CallView {
  int nsm, first_wait;
  unsigned* plan_cluster;
  Glob* glob;
  Prof* prof;
  int caller_device = -1;   // the host thread's device before, where it was another
  CallView() = default;
  CallView(const CallView&) = delete;
  CallView& operator=(const CallView&) = delete;
  ~CallView() {
    if (caller_device >= 0) cudaSetDevice(caller_device);
  }
};
int begin_call(ebc_ctx* ctx, cudaStream_t st, CallView* out);

inline int type_bytes(int type) { return type == EBC_F32 ? 4 : type == EBC_BF16 || type == EBC_F16 ? 2 : 0; }

template <typename T>
__device__ __forceinline__ float to_f32(T v);
template <>
__device__ __forceinline__ float to_f32(float v) { return v; }
template <>
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }

// round to nearest even: the one rounding of a sum that was held in fp32
template <typename T>
__device__ __forceinline__ T from_f32(float v);
template <>
__device__ __forceinline__ float from_f32(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 from_f32(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_f32(float v) { return __float2half_rn(v); }

// V bytes of a row: V / sizeof(T) elements moved by one load or store.
template <int V>
struct Raw;
template <>
struct Raw<2> {
  using T = uint16_t;
};
template <>
struct Raw<4> {
  using T = uint32_t;
};
template <>
struct Raw<8> {
  using T = uint2;
};
template <>
struct Raw<16> {
  using T = uint4;
};

template <typename T, int V>
struct Vec {
  static constexpr int kN = V / (int)sizeof(T);
  union {
    typename Raw<V>::T raw;
    T e[kN];
  };
  __device__ __forceinline__ Vec() {}
};

// Bytes per row access: the widest of 16, 8, 4 and 2 that divides every
// address given (pointers and row strides in bytes, or'ed together).
inline int vec_bytes(uintptr_t addresses, int elem) {
  for (int v = 16; v > elem; v >>= 1)
    if ((addresses & (uintptr_t)(v - 1)) == 0) return v;
  return elem;
}

// Calls f with the tag of the element type and access width.
template <typename T_, int V_>
struct Tag {
  using T = T_;
  static constexpr int V = V_;
};
template <typename T, typename F>
cudaError_t with_vec(int v, F&& f) {
  if (v == 16) return f(Tag<T, 16>{});
  if (v == 8) return f(Tag<T, 8>{});
  if constexpr (sizeof(T) == 2) {
    if (v == 4) return f(Tag<T, 4>{});
    return f(Tag<T, 2>{});
  } else {
    return f(Tag<T, 4>{});
  }
}
template <typename F>
cudaError_t with_type(int type, int v, F&& f) {
  if (type == EBC_F32) return with_vec<float>(v, f);
  if (type == EBC_BF16) return with_vec<__nv_bfloat16>(v, f);
  return with_vec<__half>(v, f);
}

// The kernels start before those ahead of them on the stream have ended (see
// pdl_enter), so what they read may still be written while they run.  Their
// inputs are therefore ordinary pointers: `const __restrict__` and __ldg would
// let the compiler use loads that take memory to be unchanged for the kernel's
// whole life, and move them ahead of the wait.
//
// Launch with cluster dimension `cluster` (1 = none) and programmatic stream
// serialization, bracketed by the profiler's events.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_named(const CallView& v, const char* name, cudaStream_t st, void (*kernel)(KArgs...),
                                dim3 grid, dim3 block, size_t smem, unsigned cluster, Args... args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = cluster;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 1 ? 2 : 1;
  prof_begin(v.prof, name, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
  prof_end(v.prof, st);
  return e;
}

inline int cuda_code(cudaError_t e) { return e == cudaSuccess ? EBC_OK : EBC_ERR_CUDA; }

}  // namespace ebc
