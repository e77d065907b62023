// ebc_mx4_product.cu -- the experts' products on 4-bit microscaled operands.
#include "ebc_mx4.cuh"

using namespace ebc;

namespace {

constexpr int kT = 16;   // rows and outputs of a tile

// Offset i >= 1, clamped to the rows and to what ascends; an offset that had to be
// clamped is the caller's error.
__device__ __forceinline__ int64_t offset_at(const int32_t* offsets, int i, int64_t floor, int64_t rows, bool* bad) {
  const int64_t v = offsets ? offsets[i] : rows;
  const int64_t c = v < floor ? floor : v > rows ? rows : v;
  if (c != v) *bad = true;
  return c;
}

// The plain kernel: a CTA takes 16 rows of one expert and 16 outputs; both
// blocks of 32 values a row go through shared memory as fp32 values, and a
// thread sums its output in fp32.  Tiles past the last expert's rows write
// zeros.
template <typename T>
__global__ void __launch_bounds__(kT* kT) k_mx4_product(const uint8_t* __restrict__ xc, const uint8_t* __restrict__ xs,
                                                        int64_t rows, int64_t width, const uint8_t* __restrict__ wc,
                                                        const uint8_t* __restrict__ ws, int64_t outs, int E,
                                                        const int32_t* __restrict__ offsets, T* __restrict__ ys,
                                                        Glob* glob) {
  pdl_enter();
  __shared__ float sx[kT][33], sw[kT][33];
  __shared__ int64_t s_r0, s_r1;
  __shared__ int s_e;
  const int tid = threadIdx.x;
  const int64_t out_tiles = (outs + kT - 1) / kT, out0 = blockIdx.x % out_tiles * kT;
  if (tid == 0) {
    // the tile-th run of 16 rows, counted expert by expert; then the rows
    // that no expert has
    int64_t tile = blockIdx.x / out_tiles, begin = 0;
    bool bad = false;
    s_e = -2;
    if (offsets && offsets[0] != 0) bad = true;
    for (int e = 0; e < E; ++e) {
      const int64_t end = offset_at(offsets, e + 1, begin, rows, &bad);
      const int64_t tiles = (end - begin + kT - 1) / kT;
      if (s_e == -2 && tile < tiles) {
        s_e = e;
        s_r0 = begin + tile * kT;
        s_r1 = s_r0 + kT < end ? s_r0 + kT : end;
      }
      if (s_e == -2) tile -= tiles;
      begin = end;
    }
    if (s_e == -2 && begin + tile * kT < rows) {
      s_e = -1;
      s_r0 = begin + tile * kT;
      s_r1 = s_r0 + kT < rows ? s_r0 + kT : rows;
    }
    if (bad) record_error(glob, EBC_ERR_INVALID_ARG);
  }
  __syncthreads();
  const int e = s_e;
  if (e == -2) return;
  const int64_t cb = EBC_MX4_CODE_BYTES(width), sb = EBC_MX4_SCALE_BYTES(width), blocks = (width + 31) / 32;
  const int i = tid / kT, o = tid % kT;
  const int64_t r = s_r0 + i, out = out0 + o;
  float acc = 0.f;
  if (e >= 0) {
    for (int64_t b = 0; b < blocks; ++b) {
      // thread (i, o) decodes byte o of row i's block, and of output i's
      const int64_t wi = out0 + i;
      float2 x2 = make_float2(0.f, 0.f), w2 = x2;
      if (r < s_r1) {
        x2 = __half22float2(mx4_values(xc[r * cb + b * 16 + o]));
        const float unit = mx4_unit(xs[r * sb + b]);
        x2.x *= unit;
        x2.y *= unit;
      }
      if (wi < outs) {
        const int64_t row = (int64_t)e * outs + wi;
        w2 = __half22float2(mx4_values(wc[row * cb + b * 16 + o]));
        const float unit = mx4_unit(ws[row * sb + b]);
        w2.x *= unit;
        w2.y *= unit;
      }
      __syncthreads();
      sx[i][2 * o] = x2.x;
      sx[i][2 * o + 1] = x2.y;
      sw[i][2 * o] = w2.x;
      sw[i][2 * o + 1] = w2.y;
      __syncthreads();
#pragma unroll
      for (int k = 0; k < 32; ++k) acc = fmaf(sx[i][k], sw[o][k], acc);
    }
  }
  if (r < s_r1 && out < outs) ys[r * outs + out] = from_f32<T>(acc);
}

bool aligned(const void* p, int bytes) { return ((uintptr_t)p & (uintptr_t)(bytes - 1)) == 0; }

template <typename T>
cudaError_t product_t(const CallView& v, const uint8_t* xc, const uint8_t* xs, int64_t rows, int64_t width,
                      const uint8_t* wc, const uint8_t* ws, int64_t outs, int E, const int32_t* offsets, void* ys,
                      cudaStream_t st) {
  const int64_t tiles = rows / kT + (E < rows ? E : rows) + 1;
  return launch_named(v, "k_mx4_product", st, k_mx4_product<T>,
                      dim3((unsigned)((outs + kT - 1) / kT * tiles)), dim3(kT * kT), 0, 1, xc, xs, rows,
                      width, wc, ws, outs, E, offsets, (T*)ys, v.glob);
}

}  // namespace

extern "C" {

int ebc_mx4_product(ebc_ctx* ctx, const uint8_t* d_x_codes, const uint8_t* d_x_scales, int64_t rows, int64_t width,
                    const uint8_t* d_w_codes, const uint8_t* d_w_scales, int64_t outs, int n_experts,
                    const int32_t* d_offsets, int out_type, void* d_ys, void* stream) {
  const int b = type_bytes(out_type);
  if (!ctx || !b || rows < 0 || rows > INT32_MAX || width < 1 || width > (1 << 24) || outs < 1 || n_experts < 1 ||
      n_experts > EBC_MAX_EXPERTS || outs > (int64_t)INT32_MAX / n_experts || (!d_offsets && n_experts != 1) ||
      !aligned(d_offsets, 4))
    return EBC_ERR_INVALID_ARG;
  if (rows > 0 && (!d_x_codes || !aligned(d_x_codes, 16) || !d_x_scales || !aligned(d_x_scales, 16) || !d_w_codes ||
                   !aligned(d_w_codes, 16) || !d_w_scales || !aligned(d_w_scales, 16) || !d_ys || !aligned(d_ys, b)))
    return EBC_ERR_INVALID_ARG;
  CallView v;
  cudaStream_t st = (cudaStream_t)stream;
  const int rc = begin_call(ctx, st, &v);
  if (rc || rows == 0) return rc;
  cudaError_t e;
  if (out_type == EBC_F32)
    e = product_t<float>(v, d_x_codes, d_x_scales, rows, width, d_w_codes, d_w_scales, outs, n_experts, d_offsets,
                         d_ys, st);
  else if (out_type == EBC_BF16)
    e = product_t<__nv_bfloat16>(v, d_x_codes, d_x_scales, rows, width, d_w_codes, d_w_scales, outs, n_experts,
                                 d_offsets, d_ys, st);
  else
    e = product_t<__half>(v, d_x_codes, d_x_scales, rows, width, d_w_codes, d_w_scales, outs, n_experts, d_offsets,
                          d_ys, st);
  return cuda_code(e);
}

}  // extern "C"
