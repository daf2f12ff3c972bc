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
  if (thin_shape(n, k)) return run_thin_linear(l, *dev, static_cast<cudaStream_t>(stream));
  Product p;
  p.type = type;
  p.M = m; p.N = k; p.K = n;
  p.A.p = X; p.A.ld = ldx;
  p.B.p = W; p.B.ld = ldw; p.B.mn_major = !w_trans;
  p.e = l.e;
  return run_product(p, *dev, static_cast<cudaStream_t>(stream));
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
  fxtx_status_t s = current_device(&dev);
  if (s != FXTX_OK) return s;
  cudaStream_t st = static_cast<cudaStream_t>(stream);

  if (m > 0 && thin_shape(n, k)) {
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
    return run_thin_grad(l, g, *dev, st);
  }
  const bool products = n > 0 && (DX || DW) && m > 0 && k > 0;
  SlopeArgs a;
  a.type = type;
  a.m = m; a.k = k;
  a.G = G; a.ldg = ldg;
  a.Z = Z; a.ldz = ldz;
  a.act = act;
  a.db = k > 0 ? DB : nullptr;
  void* ws = nullptr;
  // D is G itself where there is nothing to multiply and the products can read G where it lies
  const bool as_is = act == FXTX_ACT_NONE && type != FXTX_F32 && ((uintptr_t)G & 15u) == 0 && ldg % 8 == 0;
  const int64_t pitch = (k + 7) / 8 * 8, planes = type == FXTX_F32 ? 3 : 1;
  const size_t d_bytes = products && !as_is ? ((size_t)planes * m * pitch * 2 + 255) / 256 * 256 : 0;
  const size_t sum_bytes = a.db ? slope_ws_bytes(m, k, dev->sm_count) : 0;
  s = alloc_pooled(&ws, d_bytes + sum_bytes, st);
  if (s != FXTX_OK) return s;
  a.ws = reinterpret_cast<float*>(static_cast<char*>(ws) + d_bytes);
  if (d_bytes) {
    a.D = ws;
    a.ldd = pitch;
    a.d_planes = m * pitch;
  }
  if (a.D || a.db) s = status_of(launch_slope(a, dev->sm_count, st));

  Operand D;
  D.p = a.D ? a.D : G;
  D.ld = a.D ? a.ldd : ldg;
  D.plane_stride = a.D && type == FXTX_F32 ? a.d_planes : 0;
  if (s == FXTX_OK && DX && m > 0 && n > 0) {
    Product p;
    p.type = type;
    p.M = m; p.N = n; p.K = k;
    p.A = D;
    p.B.p = W; p.B.ld = ldw; p.B.mn_major = w_trans;
    p.e.out = DX; p.e.ldo = lddx;
    s = run_product(p, *dev, st);
  }
  if (s == FXTX_OK && DW && n > 0 && k > 0) {
    Operand x;
    x.p = X; x.ld = ldx; x.mn_major = true;
    D.mn_major = true;
    Product p;
    p.type = type;
    p.M = w_trans ? k : n; p.N = w_trans ? n : k; p.K = m;
    p.A = w_trans ? D : x;
    p.B = w_trans ? x : D;
    p.e.out = DW; p.e.ldo = lddw;
    s = run_product(p, *dev, st);
  }
  if (ws) cudaFreeAsync(ws, st);
  return s;
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
