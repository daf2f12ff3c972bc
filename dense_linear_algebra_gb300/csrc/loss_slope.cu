// loss_slope.cu — the gradient of softmax cross entropy at a product's entries (mode 2 of product_tc.cuh).
#include "product_tc.cuh"

namespace fxtx {

int* slope_error_word() { return device_error_word(); }

fxtx_status_t run_slope(fxtx_type_t type, const PlanesProduct& p, const ModeArgs<2>& x, const DeviceInfo& dev, cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return run_mode<float, 2>(p, x, dev, st);
    case FXTX_BF16: return run_mode<__nv_bfloat16, 2>(p, x, dev, st);
    default: return run_mode<__half, 2>(p, x, dev, st);
  }
}

}  // namespace fxtx
