// linear.cu — the product behind the linear layer and its gradient,
//     C_ij = sum_kk A(i, kk) B(j, kk),   out = act(C + bias_j) + R_ij:
// its operands brought into the form that the tensor copies read, and its layout over the
// tensor cores (plan_product).
#include <algorithm>
#include <cmath>

#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "linear.h"
#include "product.cuh"

namespace fxtx {
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

// Whether the tensor copies can read a 16-bit operand where it lies.
bool copyable(const Operand& o) { return ((uintptr_t)o.p & 15u) == 0 && o.ld % 8 == 0; }

// The operand's planes (rows x cols in memory), where they will lie in `at` if it has to be packed.
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

fxtx_status_t pack(const Operand& o, fxtx_type_t type, const Planes& x, const DeviceInfo& dev, cudaStream_t st) {
  PackArgs a;
  a.type = type;
  a.src = o.p;
  a.rows = x.rows;
  a.cols = x.cols;
  a.ld = o.ld;
  a.dst = const_cast<void*>(x.p);
  a.pitch = x.pitch;
  a.plane_stride = x.plane_stride;
  return status_of(launch_pack(a, dev.sm_count, st));
}

template <typename T>
fxtx_status_t run_empty(const Product& p, const DeviceInfo& dev, cudaStream_t st) {
  const int64_t blocks = std::min<int64_t>((p.M * ((p.N + 15) / 16) + 255) / 256, (int64_t)dev.sm_count * 8);
  return status_of(launch_kernel(empty_sum_kernel<T>, dim3((unsigned)blocks), 256, 0, st, p.e, p.M, p.N));
}

}  // namespace

// The layout with the least estimated time, in cycles of an SM (figures measured on GB300). A stage
// (64 of kk) takes its products (an M = 128, K = 16 product of a CTA holds the pipe for 64 cycles up
// to N = 128) or its bytes, of which an SM gets about 55 a cycle from L2 with the deep pipelines of the
// persistent kernel and a CTA of the split kernel about 32; no layout beats the operands' stream from
// HBM. A persistent CTA's tiles follow one another, each for as long as its products or its epilogue
// take. On top come a fixed cost (launch, filling the pipeline, the last epilogue) and the exchange of
// partial sums: between the CTAs of a cluster, or through memory and a second kernel.
TcPlan plan_product(int64_t M, int64_t N, int64_t K, int planes, bool a_mn, bool b_mn, int sm_count) {
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
    const double stage = std::max(mma, bytes / (cluster ? 32.0 : 55.0)), epilogue = 400.0 + 12.0 * bn;
    auto price = [&](int64_t s) {
      const int64_t per = (kb + s - 1) / s;
      if (cluster && (s - 1) * per >= kb) return;  // a CTA without work
      const int64_t waves = (tiles * s + units - 1) / units;
      double t;
      if (cluster) {
        t = std::max(floor, waves * (per * stage)) + waves * (3000.0 + 15.0 * bn) + (s > 1 ? 800.0 : 0.0);
      } else {
        t = std::max(floor, waves * std::max(per * stage, epilogue)) + 4500.0 + epilogue;
        if (s > 1) t += 4500.0 + (double)s * M * N * 8.0 / 3000.0;
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
      for (int64_t s = 1; s <= std::min<int64_t>(kb, 4 * units); s = s < 8 ? s + 1 : s + s / 4) price(s);
  };
  const int top = planes == 3 ? 64 : 128;  // the widest tile of the split kernel
  if (M <= top)
    for (int bn : {16, 32, 64, 128})
      if (bn >= M && bn <= top) consider(true, true, 1, bn);
  consider(false, true, 1, 64);
  if (planes == 1) consider(false, true, 1, 128);
  consider(false, false, 1, 64);
  consider(false, false, 1, 128);
  consider(false, false, 2, 128);
  if (planes == 1) consider(false, false, 2, 256);
  return best;
}

fxtx_status_t run_product(const Product& p, const DeviceInfo& dev, cudaStream_t st) {
  if (p.K == 0) {
    switch (p.type) {
      case FXTX_F32: return run_empty<float>(p, dev, st);
      case FXTX_BF16: return run_empty<__nv_bfloat16>(p, dev, st);
      default: return run_empty<__half>(p, dev, st);
    }
  }
  PlanesProduct q;
  q.M = p.M;
  q.N = p.N;
  q.K = p.K;
  q.e = p.e;
  size_t ab = 0, bb = 0;
  planes_of(p.A, p.type, p.M, p.K, nullptr, &ab);
  planes_of(p.B, p.type, p.N, p.K, nullptr, &bb);
  char* ws = nullptr;
  fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&ws), ab + bb, st);
  if (s != FXTX_OK) return s;
  size_t used = 0;
  q.A = planes_of(p.A, p.type, p.M, p.K, ws, &used);
  q.B = planes_of(p.B, p.type, p.N, p.K, ws + ab, &used);
  if (ab) s = pack(p.A, p.type, q.A, dev, st);
  if (s == FXTX_OK && bb) s = pack(p.B, p.type, q.B, dev, st);
  if (s == FXTX_OK) switch (p.type) {
      case FXTX_F32: s = run_planes<float>(q, dev, st); break;
      case FXTX_BF16: s = run_planes<__nv_bfloat16>(q, dev, st); break;
      default: s = run_planes<__half>(q, dev, st); break;
    }
  if (ws) cudaFreeAsync(ws, st);
  return s;
}

}  // namespace fxtx
