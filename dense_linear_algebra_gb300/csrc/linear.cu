// linear.cu — the linear layer and its gradient as products on the tensor cores,
//     C_ij = sum_kk A(i, kk) B(j, kk),   out = act(C + bias_j) + R_ij:
// operands brought into the form that the tensor copies read, where they are not in it, and
// each product's layout over the tensor cores (plan_product).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "linear.h"
#include "product.cuh"

namespace fxtx {

bool copyable(const Operand& o) { return ((uintptr_t)o.p & 15u) == 0 && o.ld % 8 == 0; }

Planes planes_of(const Operand& o, fxtx_type_t type, int64_t mn, int64_t k, char* at, size_t* bytes) {
  Planes x;
  x.rows = o.mn_major ? k : mn;
  x.cols = o.mn_major ? mn : k;
  x.mn_major = o.mn_major;
  x.planes = type == FXTX_F32 ? 3 : 1;
  *bytes = 0;
  if (o.plane_stride > 0 || (type != FXTX_F32 && copyable(o))) {
    x.p = o.p;
    x.pitch = o.ld;
    x.plane_stride = o.plane_stride > 0 ? o.plane_stride : x.rows * x.pitch;
  } else {
    x.p = at;
    x.pitch = (x.cols + 7) / 8 * 8;
    x.plane_stride = x.rows * x.pitch;
    *bytes = ((size_t)x.planes * x.plane_stride * 2 + 255) / 256 * 256;
  }
  return x;
}

namespace {

// A sum of no terms: out = act(bias_j) + R_ij.
template <typename T>
__global__ void __launch_bounds__(256) empty_sum_kernel(const Epilogue e, int64_t rows, int64_t cols) {
  const Finish<T> fin(e, rows, cols);
  const int64_t groups = (cols + 15) / 16, stride = (int64_t)gridDim.x * 256;
  const float zero[16] = {};
  after_previous();
  for (int64_t x = (int64_t)blockIdx.x * 256 + threadIdx.x; x < rows * groups; x += stride)
    fin.template row<16>(x / groups, x % groups * 16, zero);
}

fxtx_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

// Up to two operands and what has to be copied for them, in one workspace.
struct Prepared {
  fxtx_type_t type;
  PackArgs packs[2];
  int count = 0;
  size_t bytes = 0;
  size_t at[2];        // the copies' places in the workspace
  Planes* of[2];       // and whose they are

  Planes add(const Operand& o, int64_t mn, int64_t k, Planes* slot) {
    size_t need = 0;
    *slot = planes_of(o, type, mn, k, nullptr, &need);
    if (need) {
      PackArgs& a = packs[count];
      a.src = o.p;
      a.rows = slot->rows;
      a.cols = slot->cols;
      a.ld = o.ld;
      a.pitch = slot->pitch;
      a.plane_stride = slot->plane_stride;
      at[count] = bytes;
      of[count++] = slot;
      bytes += need;
    }
    return *slot;
  }
  // once the workspace is there
  void place(char* ws) {
    for (int i = 0; i < count; ++i) of[i]->p = packs[i].dst = ws + at[i];
  }
};

fxtx_status_t run_typed(fxtx_type_t type, const PlanesProduct& q, const DeviceInfo& dev, cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return run_planes<float>(q, dev, st);
    case FXTX_BF16: return run_planes<__nv_bfloat16>(q, dev, st);
    default: return run_planes<__half>(q, dev, st);
  }
}

template <typename T>
cudaError_t empty_t(const Epilogue& e, int64_t rows, int64_t cols, const DeviceInfo& dev, cudaStream_t st) {
  const int64_t blocks = std::min<int64_t>((rows * ((cols + 15) / 16) + 255) / 256, (int64_t)dev.sm_count * 8);
  return launch_kernel(empty_sum_kernel<T>, dim3((unsigned)blocks), 256, 0, st, e, rows, cols);
}
fxtx_status_t run_empty(fxtx_type_t type, const Epilogue& e, int64_t rows, int64_t cols, const DeviceInfo& dev,
                        cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return status_of(empty_t<float>(e, rows, cols, dev, st));
    case FXTX_BF16: return status_of(empty_t<__nv_bfloat16>(e, rows, cols, dev, st));
    default: return status_of(empty_t<__half>(e, rows, cols, dev, st));
  }
}

}  // namespace

// The layout with the least estimated time, in cycles of an SM (figures measured on GB300). A stage
// (64 of kk) takes its products (an M = 128, K = 16 product of a CTA holds the pipe for 64 cycles up
// to N = 128) or its bytes, of which an SM gets about 55 a cycle from L2 with the deep pipelines of the
// persistent kernel and a CTA of the split kernel 27 to 34; no layout beats the operands' stream from
// HBM. A persistent CTA's tiles follow one another, each for as long as its products or its epilogue
// take. On top come a fixed cost (launch, filling the pipeline, the last epilogue) and the exchange of
// partial sums: between the CTAs of a cluster, or through memory and a second kernel.
static TcPlan best_plan(int64_t M, int64_t N, int64_t K, int planes, bool a_mn, bool b_mn, int sm_count, bool clusters,
                        int64_t most) {
  TcPlan best;
  double best_t = 1e300;
  const double floor = planes * 2.0 * K * (double)(M + N) / 3400.0;
  auto consider = [&](bool swap, bool cluster, int cg, int bn) {
    const int64_t L = swap ? N : M, Cn = swap ? M : N;
    if ((swap ? a_mn : b_mn) && bn / cg < 64) return;  // an MN-major box is 64 wide
    const int64_t tiles = ((L + 128 * cg - 1) / (128 * cg)) * ((Cn + bn - 1) / bn);
    // CTAs (or pairs) at a time: two of the split kernel's narrow ones share an SM
    const int64_t units = cluster && planes == 1 && bn <= 64 ? 2 * sm_count : sm_count / cg;
    const int bk = planes == 1 && !cluster ? 128 : 64;  // kk a stage
    const int64_t kb = std::max<int64_t>(1, (K + bk - 1) / bk);
    const double mma = bk / 16 * (planes == 3 ? 6 : 1) * std::max(64.0, bn / 2.0);
    const double bytes = planes * 2.0 * bk * (128.0 + bn / cg);
    const double stage = std::max(mma, bytes / (!cluster ? 55.0 : bn <= 64 ? 27.0 : 34.0)), epilogue = 400.0 + 12.0 * bn;
    auto price = [&](int64_t s) {
      const int64_t per = (kb + s - 1) / s;
      if (cluster && (s - 1) * per >= kb) return;  // a CTA without work
      const int64_t waves = (tiles * s + units - 1) / units;
      double t;
      if (cluster) {
        t = std::max(floor, waves * (per * stage)) + waves * (3500.0 + 15.0 * bn) + (s > 1 ? 800.0 : 0.0);
      } else {
        t = std::max(floor, waves * std::max(per * stage, epilogue)) + 3000.0 + epilogue;
        if (s > 1) t += 6500.0 + (double)s * M * N * 8.0 / 3000.0;
      }
      if (t < best_t) {
        best_t = t;
        best.swap = swap;
        best.cluster = cluster;
        best.cg = cg;
        best.bn = bn;
        best.splits = (int)s;
      }
    };
    if (cluster)
      for (int s = 1; s <= 8; s *= 2) price(s);
    else
      for (int64_t s = 1; s <= std::min<int64_t>({kb, 4 * units, most}); s = s < 8 ? s + 1 : s + s / 4) price(s);
  };
  const int top = planes == 3 ? 64 : 128;  // the widest tile of the split kernel
  if (clusters) {
    if (M <= top)
      for (int bn : {16, 32, 64, 128})
        if (bn >= M && bn <= top) consider(true, true, 1, bn);
    consider(false, true, 1, 64);
    if (planes == 1) consider(false, true, 1, 128);
  }
  consider(false, false, 1, 64);
  consider(false, false, 1, 128);
  consider(false, false, 2, 128);
  if (planes == 1) consider(false, false, 2, 256);
  return best;
}

TcPlan plan_product(int64_t M, int64_t N, int64_t K, int planes, bool a_mn, bool b_mn, int sm_count) {
  return best_plan(M, N, K, planes, a_mn, b_mn, sm_count, true, INT64_MAX);
}
TcPlan plan_persistent(int64_t M, int64_t N, int64_t K, int planes, bool a_mn, bool b_mn, int sm_count, int64_t splits) {
  return best_plan(M, N, K, planes, a_mn, b_mn, sm_count, false, splits);
}

// Whether a result of m rows is formed on the CUDA cores.
bool few_rows(fxtx_type_t type, int64_t m, bool by_column) {
  return type == FXTX_F32 && m <= (by_column ? kFewByColumn : kFewByRow);
}

fxtx_status_t run_linear(const LayerArgs& l, const DeviceInfo& dev, cudaStream_t st) {
  if (l.n == 0) return run_empty(l.type, l.e, l.m, l.k, dev, st);
  if (few_rows(l.type, l.m, l.w_trans))
    return run_few(l.m, l.n, l.k, l.X, l.ldx, 0, static_cast<const float*>(l.W), l.ldw, l.w_trans, l.e, dev, st);
  Operand x, w;
  x.p = l.X; x.ld = l.ldx;
  w.p = l.W; w.ld = l.ldw; w.mn_major = !l.w_trans;
  PlanesProduct q;
  q.M = l.m;
  q.N = l.k;
  q.K = l.n;
  q.e = l.e;
  Prepared p;
  p.type = l.type;
  p.add(x, l.m, l.n, &q.A);
  p.add(w, l.k, l.n, &q.B);
  char* ws = nullptr;
  fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&ws), p.bytes, st);
  if (s != FXTX_OK) return s;
  p.place(ws);
  s = status_of(launch_prepare(l.type, nullptr, p.packs, p.count, dev.sm_count, st));
  if (s == FXTX_OK) s = run_typed(l.type, q, dev, st);
  if (ws) cudaFreeAsync(ws, st);
  return s;
}

fxtx_status_t run_grad(const LayerArgs& l, const GradArgs& g, const DeviceInfo& dev, cudaStream_t st) {
  const bool dx = g.DX && l.m > 0 && l.n > 0, dw = g.DW && l.n > 0 && l.k > 0, f32 = l.type == FXTX_F32;
  const bool sums = l.m > 0 && l.k > 0;  // a sum of no terms is zero
  // D is G itself where there is nothing to multiply and the products can read G where it lies
  Operand d;
  d.p = g.G; d.ld = g.ldg;
  const bool own = sums && (dx || dw) && (g.act != FXTX_ACT_NONE || f32 || !copyable(d));
  SlopeArgs a;
  a.m = l.m; a.k = l.k;
  a.G = g.G; a.ldg = g.ldg;
  a.Z = g.Z; a.ldz = g.ldz;
  a.act = g.act;
  a.db = l.k > 0 ? g.DB : nullptr;

  Prepared p;
  p.type = l.type;
  PlanesProduct qx, qw;
  const bool few = few_rows(l.type, l.m, !l.w_trans);  // dX = D W^T takes W in the other order
  if (sums && dx && !few) {
    Operand w;
    w.p = l.W; w.ld = l.ldw; w.mn_major = l.w_trans;
    qx.M = l.m; qx.N = l.n; qx.K = l.k;
    p.add(w, l.n, l.k, &qx.B);
  }
  Planes xp;
  if (sums && dw) {
    Operand x;
    x.p = l.X; x.ld = l.ldx; x.mn_major = true;
    qw.M = l.w_trans ? l.k : l.n; qw.N = l.w_trans ? l.n : l.k; qw.K = l.m;
    p.add(x, l.n, l.m, &xp);
  }
  const size_t d_at = p.bytes, pitch = (size_t)(l.k + 7) / 8 * 8;
  const size_t d_bytes = own ? ((size_t)(f32 ? 3 : 1) * l.m * pitch * 2 + 255) / 256 * 256 : 0;
  const size_t sum_bytes = a.db ? slope_ws_bytes(l.m, l.k, dev.sm_count) : 0;
  char* ws = nullptr;
  fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&ws), d_at + d_bytes + sum_bytes, st);
  if (s != FXTX_OK) return s;
  p.place(ws);
  a.ws = reinterpret_cast<float*>(ws + d_at + d_bytes);
  if (own) {
    a.D = ws + d_at;
    a.ldd = (int64_t)pitch;
    a.d_planes = l.m * (int64_t)pitch;
    d.p = a.D;
    d.ld = a.ldd;
    d.plane_stride = f32 ? a.d_planes : 0;
  }
  s = status_of(launch_prepare(l.type, own || a.db ? &a : nullptr, p.packs, p.count, dev.sm_count, st));

  size_t none = 0;
  Epilogue e;
  if (s == FXTX_OK && dx) {
    e.out = g.DX;
    e.ldo = g.lddx;
    if (sums && few) {
      s = run_few(l.m, l.k, l.n, d.p, d.ld, d.plane_stride, static_cast<const float*>(l.W), l.ldw, !l.w_trans, e, dev, st);
    } else if (sums) {
      qx.A = planes_of(d, l.type, l.m, l.k, nullptr, &none);
      qx.e = e;
      s = run_typed(l.type, qx, dev, st);
    } else {
      s = run_empty(l.type, e, l.m, l.n, dev, st);
    }
  }
  if (s == FXTX_OK && dw) {
    e.out = g.DW;
    e.ldo = g.lddw;
    const int64_t rows = l.w_trans ? l.k : l.n, cols = l.w_trans ? l.n : l.k;
    if (sums) {
      d.mn_major = true;
      const Planes dp = planes_of(d, l.type, l.k, l.m, nullptr, &none);
      qw.A = l.w_trans ? dp : xp;
      qw.B = l.w_trans ? xp : dp;
      qw.e = e;
      s = run_typed(l.type, qw, dev, st);
    } else {
      s = run_empty(l.type, e, rows, cols, dev, st);
    }
  }
  if (ws) cudaFreeAsync(ws, st);
  return s;
}

}  // namespace fxtx
