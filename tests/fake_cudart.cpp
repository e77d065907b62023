// A CUDA runtime without a device, for the tests of what the library does on
// the host: the library's objects are linked with this file instead of the CUDA
// runtime.  Device memory is host memory, streams and events are only names,
// nothing is executed; calls of interest are written into a log that the test
// reads, and a launch may be handed to the test, which can do the kernel's work.
//
// The rules of the runtime that the tests are about are kept: a current device
// per host thread; a cluster of more than 8 has to be allowed and to fit; and a
// launch fails when its dynamic and static shared memory
// pass 48 KB and the kernel's attribute does not allow it.
#include <cuda_runtime_api.h>

#include <chrono>
#include <cstdarg>
#include <cstdio>
#include <cstdlib>
#include <cstring>
#include <map>
#include <mutex>
#include <string>
#include <thread>

extern "C" {
typedef void (*fake_launch_cb)(const char* name, void** args);
}

namespace {
std::recursive_mutex g_lock;   // of the log and the maps
std::string g_log;
std::map<const void*, std::string> g_kernels;        // host function -> device name
std::map<const void*, int> g_shared_limit;           // host function -> dynamic shared memory allowed
std::map<const void*, int> g_large_cluster;          // host function -> clusters of more than 8 allowed
fake_launch_cb g_on_launch = nullptr;
int g_static_shared = 256, g_max_clusters = 8;
thread_local int g_device = 0;

void logf(const char* format, ...) {
  char line[512];
  va_list v;
  va_start(v, format);
  vsnprintf(line, sizeof line, format, v);
  va_end(v);
  std::lock_guard<std::recursive_mutex> hold(g_lock);
  g_log += line;
  g_log += '\n';
}
const char* name_of(const void* f) {
  auto it = g_kernels.find(f);
  return it == g_kernels.end() ? "?" : it->second.c_str();
}
}  // namespace

extern "C" {

// ---- what the tests call ----
const char* fake_log() { return g_log.c_str(); }
void fake_clear() { g_log.clear(); }
void fake_on_launch(fake_launch_cb cb) { g_on_launch = cb; }
void fake_static_shared(int bytes) { g_static_shared = bytes; }
void fake_max_clusters(int n) { g_max_clusters = n; }

// ---- registration, as the compiler's host code makes it ----
void** __cudaRegisterFatBinary(void* f) { return (void**)f; }
void __cudaRegisterFatBinaryEnd(void**) {}
void __cudaUnregisterFatBinary(void**) {}
void __cudaRegisterFunction(void**, const char* host, char*, const char* name, int, uint3*, uint3*, dim3*, dim3*, int*) {
  g_kernels[host] = name;
}
void __cudaRegisterVar(void**, char*, char*, const char*, int, size_t, int, int) {}
cudaError_t __cudaGetKernel(cudaKernel_t* k, const void* host) {
  *k = (cudaKernel_t)host;
  return cudaSuccess;
}
cudaError_t __cudaLaunchKernel(cudaKernel_t, dim3, dim3, void**, size_t, cudaStream_t) { return cudaErrorNotSupported; }
cudaError_t __cudaPopCallConfiguration(dim3*, dim3*, size_t*, void*) { return cudaErrorNotSupported; }

// ---- devices ----
cudaError_t cudaGetDeviceCount(int* n) {
  *n = 2;
  return cudaSuccess;
}
cudaError_t cudaGetDevice(int* d) {
  *d = g_device;
  return cudaSuccess;
}
cudaError_t cudaSetDevice(int d) {
  if (d < 0 || d > 1) return cudaErrorInvalidDevice;
  g_device = d;
  return cudaSuccess;
}
cudaError_t cudaGetDeviceProperties(cudaDeviceProp* p, int) {
  memset(p, 0, sizeof *p);
  p->major = 10;
  p->minor = 3;
  p->multiProcessorCount = 152;
  return cudaSuccess;
}
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr, int) {
  *v = 152;
  return cudaSuccess;
}
cudaError_t cudaDeviceSynchronize() {
  logf("sync device %d", g_device);
  return cudaSuccess;
}
cudaError_t cudaGetLastError() { return cudaSuccess; }

// ---- memory ----
cudaError_t cudaMalloc(void** p, size_t n) {
  *p = calloc(1, n ? n : 1);
  return cudaSuccess;
}
cudaError_t cudaFree(void* p) {
  free(p);
  return cudaSuccess;
}
cudaError_t cudaHostAlloc(void** p, size_t n, unsigned) { return cudaMalloc(p, n); }
cudaError_t cudaFreeHost(void* p) { return cudaFree(p); }
cudaError_t cudaMemset(void* p, int v, size_t n) {
  memset(p, v, n);
  return cudaSuccess;
}
cudaError_t cudaMemsetAsync(void* p, int v, size_t n, cudaStream_t) { return cudaMemset(p, v, n); }
cudaError_t cudaMemcpy(void* d, const void* s, size_t n, cudaMemcpyKind kind) {
  logf("copy %s %zu", kind == cudaMemcpyDeviceToHost ? "to host" : "to device", n);
  memcpy(d, s, n);
  return cudaSuccess;
}
cudaError_t cudaMemcpyAsync(void* d, const void* s, size_t n, cudaMemcpyKind kind, cudaStream_t) {
  return cudaMemcpy(d, s, n, kind);
}
cudaError_t cudaGetSymbolAddress(void**, const void*) { return cudaErrorNotSupported; }

// ---- streams and events ----
cudaError_t cudaStreamSynchronize(cudaStream_t s) {
  logf("sync stream %p", (void*)s);
  return cudaSuccess;
}
cudaError_t cudaEventCreate(cudaEvent_t* e) {
  *e = (cudaEvent_t)malloc(1);
  return cudaSuccess;
}
cudaError_t cudaEventDestroy(cudaEvent_t e) {
  free(e);
  return cudaSuccess;
}
cudaError_t cudaEventRecord(cudaEvent_t, cudaStream_t) { return cudaSuccess; }
cudaError_t cudaEventSynchronize(cudaEvent_t) { return cudaSuccess; }
cudaError_t cudaEventElapsedTime(float* ms, cudaEvent_t, cudaEvent_t) {
  *ms = 1.f;
  return cudaSuccess;
}

// ---- kernels ----
cudaError_t cudaFuncSetAttribute(const void* f, cudaFuncAttribute a, int v) {
  std::lock_guard<std::recursive_mutex> hold(g_lock);
  if (a == cudaFuncAttributeMaxDynamicSharedMemorySize) {
    g_shared_limit[f] = v;
    logf("shared %s %d", name_of(f), v);
  }
  if (a == cudaFuncAttributeNonPortableClusterSizeAllowed) g_large_cluster[f] = v;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveBlocksPerMultiprocessorWithFlags(int* n, const void*, int, size_t, unsigned) {
  *n = 2;
  return cudaSuccess;
}
cudaError_t cudaOccupancyMaxActiveClusters(int* n, const void*, const cudaLaunchConfig_t*) {
  *n = g_max_clusters;
  return cudaSuccess;
}
cudaError_t cudaLaunchKernelExC(const cudaLaunchConfig_t* c, const void* f, void** args) {
  std::lock_guard<std::recursive_mutex> hold(g_lock);
  unsigned cluster = 1;
  for (unsigned i = 0; i < c->numAttrs; ++i)
    if (c->attrs[i].id == cudaLaunchAttributeClusterDimension) cluster = c->attrs[i].val.clusterDim.x;
  auto it = g_shared_limit.find(f);
  const size_t allowed = it == g_shared_limit.end() ? 0 : (size_t)it->second;
  const bool fits = c->dynamicSmemBytes + g_static_shared <= (allowed > 48 * 1024 ? allowed + 1024 : 48 * 1024) &&
                    (cluster <= 8 || (g_large_cluster[f] && g_max_clusters > 0));
  logf("launch %s grid %u cluster %u shared %zu stream %p device %d%s", name_of(f), c->gridDim.x, cluster,
       c->dynamicSmemBytes, (void*)c->stream, g_device, fits ? "" : " refused");
  if (!fits) return cudaErrorInvalidValue;
  if (g_on_launch) g_on_launch(name_of(f), args);
  return cudaSuccess;
}
// cuTensorMapEncodeTiled is the one entry point that is asked for
static int fake_encode(void*, int, unsigned, void*, const void*, const void*, const void*, const void*, int, int, int, int) {
  return 0;
}
cudaError_t cudaGetDriverEntryPointByVersion(const char* name, void** p, unsigned, unsigned long long,
                                             cudaDriverEntryPointQueryResult* q) {
  logf("entry point %s", name);
  std::this_thread::sleep_for(std::chrono::milliseconds(50));   // other threads may ask meanwhile
  *p = (void*)fake_encode;
  *q = cudaDriverEntryPointSuccess;
  return cudaSuccess;
}

}  // extern "C"
