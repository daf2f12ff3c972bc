// layers_api.cu — the C entry points of the layer operators (declared in include/fxtx.h):
// argument checks, workspace and the launches, all enqueued on the caller's stream.
#include <cmath>

#include "host.h"
#include "layers.h"
#include "linear.h"

using namespace fxtx;

namespace {

fxtx_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

// A matrix argument with `rows` rows of `cols` entries: its pitch, and its pointer where it has entries.
bool rows_ok(const void* p, int64_t rows, int64_t cols, int64_t ld) {
  return ld >= cols && (p != nullptr || rows == 0 || cols == 0);
}

// Sizes the kernels index: every matrix within 2^46 entries, each size within 2^31.
bool sizes_ok(int64_t m, int64_t n, int64_t k) {
  const int64_t top = (int64_t)1 << 31;
  return m >= 0 && n >= 0 && k >= 0 && m < top && n < top && k < top;
}

}  // namespace

extern "C" {

fxtx_status_t fxtx_linear(fxtx_type_t type, int64_t m, int64_t n, int64_t k, const void* X, int64_t ldx, const void* W,
                          int64_t ldw, int w_trans, const void* b, fxtx_act_t act, const void* R, int64_t ldr, void* Z,
                          int64_t ldz, void* OUT, int64_t ldo, void* stream) {
  if (!type_ok(type) || !act_ok(act) || !sizes_ok(m, n, k) || (w_trans != 0 && w_trans != 1)) return FXTX_ERR_INVALID_ARG;
  if (!rows_ok(X, m, n, ldx) || !rows_ok(W, w_trans ? k : n, w_trans ? n : k, ldw) || !rows_ok(OUT, m, k, ldo))
    return FXTX_ERR_INVALID_ARG;
  if ((R != nullptr && ldr < k) || (Z != nullptr && ldz < k)) return FXTX_ERR_INVALID_ARG;
  if (m == 0 || k == 0) return FXTX_OK;
  const DeviceInfo* dev = nullptr;
  const fxtx_status_t s = current_device(&dev);
  if (s != FXTX_OK) return s;
  LayerArgs l;
  l.type = type;
  l.m = m; l.n = n; l.k = k;
  l.X = X; l.ldx = ldx;
  l.W = W; l.ldw = ldw; l.w_trans = w_trans != 0;
  l.e.bias = b; l.e.act = act;
  l.e.R = R; l.e.ldr = ldr;
  l.e.Z = Z; l.e.ldz = ldz;
  l.e.out = OUT; l.e.ldo = ldo;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return thin_shape(n, k) ? run_thin_linear(l, *dev, st) : run_linear(l, *dev, st);
}

fxtx_status_t fxtx_linear_grad(fxtx_type_t type, int64_t m, int64_t n, int64_t k, const void* G, int64_t ldg,
                               const void* X, int64_t ldx, const void* W, int64_t ldw, int w_trans, const void* Z,
                               int64_t ldz, fxtx_act_t act, void* DX, int64_t lddx, void* DW, int64_t lddw, void* DB,
                               void* stream) {
  if (!type_ok(type) || !act_ok(act) || !sizes_ok(m, n, k) || (w_trans != 0 && w_trans != 1)) return FXTX_ERR_INVALID_ARG;
  if (!rows_ok(G, m, k, ldg)) return FXTX_ERR_INVALID_ARG;
  if (act != FXTX_ACT_NONE && !rows_ok(Z, m, k, ldz)) return FXTX_ERR_INVALID_ARG;
  if (DX && (!rows_ok(W, w_trans ? k : n, w_trans ? n : k, ldw) || lddx < n)) return FXTX_ERR_INVALID_ARG;
  if (DW && (!rows_ok(X, m, n, ldx) || lddw < (w_trans ? n : k))) return FXTX_ERR_INVALID_ARG;
  if ((n == 0 || (!DX && !DW)) && (!DB || k == 0)) return FXTX_OK;
  const DeviceInfo* dev = nullptr;
  const fxtx_status_t s = current_device(&dev);
  if (s != FXTX_OK) return s;
  LayerArgs l;
  l.type = type;
  l.m = m; l.n = n; l.k = k;
  l.X = X; l.ldx = ldx;
  l.W = W; l.ldw = ldw; l.w_trans = w_trans != 0;
  GradArgs g;
  g.G = G; g.ldg = ldg;
  g.Z = Z; g.ldz = ldz;
  g.act = act;
  g.DX = DX; g.lddx = lddx;
  g.DW = DW; g.lddw = lddw;
  g.DB = DB;
  cudaStream_t st = static_cast<cudaStream_t>(stream);
  return m > 0 && thin_shape(n, k) ? run_thin_grad(l, g, *dev, st) : run_grad(l, g, *dev, st);
}

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
