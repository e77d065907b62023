// ebc_mx4_product.cu -- the experts' products on 4-bit microscaled operands
// (the kernels' common part is in ebc_mx_product.cuh).
#include "ebc_mx_product.cuh"

namespace {

template <int kTN, int kCtas>
__global__ void __launch_bounds__(kThreads, 1) k_mx4_product(const __grid_constant__ CUtensorMap wmap,
                                                             const __grid_constant__ CUtensorMap xmap, Args a) {
  __shared__ Shared<Geom<Mx4Format, kTN, kCtas>> sh;
  product_begin<Mx4Format, kTN, kCtas>(sh);
  pdl_enter();
  product_run<Mx4Format, kTN, kCtas>(sh, wmap, xmap, a);
}

struct Mx4Launch {
  using Format = Mx4Format;
  template <int kTN, int kCtas>
  static constexpr auto kernel() {
    return k_mx4_product<kTN, kCtas>;
  }
};

}  // namespace

extern "C" {

int ebc_mx4_product(ebc_ctx* ctx, const uint8_t* d_x_codes, const uint8_t* d_x_scales, int64_t rows, int64_t width,
                    const uint8_t* d_w_codes, const uint8_t* d_w_scales, int64_t outs, int n_experts,
                    const int32_t* d_offsets, int out_type, void* d_ys, void* stream) {
  return product_any<Mx4Launch>(ctx, d_x_codes, d_x_scales, rows, width, d_w_codes, d_w_scales, outs, n_experts,
                                d_offsets, out_type, d_ys, stream);
}

}  // extern "C"
