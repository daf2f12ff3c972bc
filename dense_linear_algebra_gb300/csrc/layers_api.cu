// layers_api.cu — the C entry points of the layer operators (declared in include/fxtx.h):
// argument checks, workspace and the launches, all enqueued on the caller's stream.
#include <cmath>

#include "host.h"
#include "layers.h"

using namespace fxtx;

namespace {

fxtx_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

}  // namespace

extern "C" {

fxtx_status_t fxtx_adamw(int64_t count, const fxtx_adamw_tensor_t* tensors, fxtx_type_t p_type, fxtx_type_t g_type,
                         fxtx_type_t copy_type, int state_bits, int64_t step, double lr, double beta1, double beta2,
                         double eps, double weight_decay, void* stream) {
  if (count < 0 || step < 1 || !type_ok(p_type) || !type_ok(g_type) || !type_ok(copy_type) ||
      (state_bits != 8 && state_bits != 32))
    return FXTX_ERR_INVALID_ARG;
  // written so that a NaN is refused
  if (!(beta1 >= 0.0 && beta1 < 1.0) || !(beta2 >= 0.0 && beta2 < 1.0) || !(eps >= 0.0) || !(lr >= 0.0) ||
      !(weight_decay >= 0.0) || !std::isfinite(lr) || !std::isfinite(eps) || !std::isfinite(weight_decay))
    return FXTX_ERR_INVALID_ARG;
  if (count > 0 && tensors == nullptr) return FXTX_ERR_INVALID_ARG;
  bool any = false;
  for (int64_t i = 0; i < count; ++i) {
    const fxtx_adamw_tensor_t& t = tensors[i];
    if (t.n < 0 || t.n > ((int64_t)1 << 39)) return FXTX_ERR_INVALID_ARG;
    if (t.n == 0) continue;
    any = true;
    if (!t.p || !t.g || !t.m || !t.v || (state_bits == 8 && (!t.m_scale || !t.v_scale))) return FXTX_ERR_INVALID_ARG;
  }
  if (!any) return FXTX_OK;
  const DeviceInfo* dev = nullptr;
  const fxtx_status_t s = current_device(&dev);
  if (s != FXTX_OK) return s;
  AdamwConst c;
  c.b1 = (float)beta1;
  c.c1 = (float)(1.0 - beta1);
  c.b2 = (float)beta2;
  c.c2 = (float)(1.0 - beta2);
  c.root = (float)(1.0 / std::sqrt(1.0 - std::pow(beta2, (double)step)));
  c.eps = (float)eps;
  c.keep = (float)(1.0 - lr * weight_decay);
  c.rate = (float)(lr / (1.0 - std::pow(beta1, (double)step)));
  return status_of(launch_adamw(count, tensors, p_type, g_type, copy_type, state_bits, c, dev->sm_count,
                                static_cast<cudaStream_t>(stream)));
}

fxtx_status_t fxtx_adamw_moments(int64_t n, const int8_t* m, const float* m_scale, const uint8_t* v,
                                 const float* v_scale, float* m_out, float* v_out, void* stream) {
  if (n < 0 || n > ((int64_t)1 << 39)) return FXTX_ERR_INVALID_ARG;
  if (n == 0) return FXTX_OK;
  if (!m || !m_scale || !v || !v_scale || !m_out || !v_out) return FXTX_ERR_INVALID_ARG;
  const DeviceInfo* dev = nullptr;
  const fxtx_status_t s = current_device(&dev);
  if (s != FXTX_OK) return s;
  return status_of(
      launch_adamw_moments(n, m, m_scale, v, v_scale, m_out, v_out, static_cast<cudaStream_t>(stream)));
}

}  // extern "C"
