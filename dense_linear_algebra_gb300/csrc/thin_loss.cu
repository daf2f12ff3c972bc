// thin_loss.cu — softmax cross entropy on a linear layer of at most 64 features and classes, and its gradient, on the
// kernels' parts of thin.cu: a warp forms 16 rows' Z = X W + b in registers, a row's classes in one quad of lanes, so that
// its largest, its sum of exponentials and its label's entry take two exchanges each, and X is read once.
//
// Bound: HBM (X), then the latency of few warps where dW is summed.
#include "thin.cuh"

namespace fxtx {
namespace {

template <typename T, int KN, int KC>
__global__ void __launch_bounds__(THREADS) thin_loss_kernel(const __grid_constant__ ThinArgs a) {
  __shared__ uint2 ws[KN * (2 * KC) * Term<T>::P * 32];
  __shared__ float s_bias[16 * KC];
  after_previous();
  stage_operand<T, KN, 2 * KC>(ws, static_cast<const T*>(a.W), a.ws0, a.ws1, a.n, a.k);
  stage_bias<T, KC>(s_bias, a);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t tiles = (a.m + 15) / 16, step = (int64_t)gridDim.x * WARPS;
  const Rows<T, KN> rows(a.X, a.ldx, a.n);
  int64_t w = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  Chunk<T, KN> next;
  rows.load(w * 16, a.m, next);
  __syncthreads();
  for (; w < tiles; w += step) {
    const Chunk<T, KN> x = next;
    float z[2][4 * KC];
    rows.load((w + step) * 16, a.m, next);
    rows_times<T, KN, 2 * KC>(x, ws, z);
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int64_t r = w * 16 + g + 8 * h;
      const int64_t label = r < a.m ? label_at(a.loss.labels, a.loss.labels64, r, a.k) : -1;
      const int at = (int)label - 4 * KC * t;
      float top = -INFINITY, target = 0.f, sum = 0.f;
#pragma unroll
      for (int i = 0; i < 4 * KC; ++i) {
        z[h][i] += s_bias[4 * KC * t + i];
        top = fmaxf(top, z[h][i]);
        if (i == at && label >= 0) target = z[h][i];
      }
      top = fmaxf(top, shfl_xor(top, 1));
      top = fmaxf(top, shfl_xor(top, 2));
      const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
      for (int i = 0; i < 4 * KC; ++i) sum += exp_of<T>(z[h][i] - from);
      sum = group_sum<4>(sum);
      target = group_sum<4>(target);
      if (t == 0 && r < a.m) {
        const float rest = logf(sum);
        if (a.loss.loss) a.loss.loss[r] = label >= 0 ? (from - target) + rest : 0.f;
        if (a.loss.lse) a.loss.lse[r] = from + rest;
      }
    }
  }
}

template <typename T, int KN, int KC>
cudaError_t launch_loss(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return launch_kernel(thin_loss_kernel<T, KN, KC>, dim3(grid_of<thin_loss_kernel<T, KN, KC>>(a.m, sm_count)), THREADS, 0, st, a);
}
template <typename T, int KN>
cudaError_t loss_k(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return a.k <= 16 ? launch_loss<T, KN, 1>(a, sm_count, st)
                   : a.k <= 32 ? launch_loss<T, KN, 2>(a, sm_count, st) : launch_loss<T, KN, 4>(a, sm_count, st);
}
template <typename T>
cudaError_t loss_t(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return a.n <= 16 ? loss_k<T, 1>(a, sm_count, st)
                   : a.n <= 32 ? loss_k<T, 2>(a, sm_count, st) : loss_k<T, 4>(a, sm_count, st);
}

ThinArgs thin_args(const LayerArgs& l, const LossArgs& q) {
  ThinArgs a = {};
  a.m = l.m;
  a.n = (int)l.n;
  a.k = (int)l.k;
  a.X = l.X;
  a.ldx = l.ldx;
  a.W = l.W;
  a.ws0 = l.w_trans ? 1 : l.ldw;
  a.ws1 = l.w_trans ? l.ldw : 1;
  a.e = l.e;
  a.loss = q;
  return a;
}

}  // namespace

fxtx_status_t run_thin_loss(const LayerArgs& l, const LossArgs& q, const DeviceInfo& dev, cudaStream_t st) {
  const ThinArgs a = thin_args(l, q);
  cudaError_t e;
  switch (l.type) {
    case FXTX_F32: e = loss_t<float>(a, dev.sm_count, st); break;
    case FXTX_BF16: e = loss_t<__nv_bfloat16>(a, dev.sm_count, st); break;
    default: e = loss_t<__half>(a, dev.sm_count, st); break;
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

fxtx_status_t run_thin_loss_grad(const LayerArgs& l, const LossArgs& q, const DeviceInfo& dev, cudaStream_t st) {
  ThinArgs a = thin_args(l, q);
  a.DX = q.DX;
  a.lddx = q.lddx;
  a.DW = q.DW;
  a.dws0 = l.w_trans ? 1 : q.lddw;
  a.dws1 = l.w_trans ? q.lddw : 1;
  a.DB = q.DB;
  float* scales = nullptr;
  if (l.type == FXTX_F16) {
    const fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&scales), kScaleBytes, st);
    if (s != FXTX_OK) return s;
    if (launch_scales(q, l.m, l.k, scales, st) != cudaSuccess) {
      cudaGetLastError();
      cudaFreeAsync(scales, st);
      return FXTX_ERR_CUDA;
    }
    a.scales = scales;
  }
  fxtx_status_t s;
  switch (l.type) {
    case FXTX_F32: s = grad_t<float, true>(a, dev.sm_count, st); break;
    case FXTX_BF16: s = grad_t<__nv_bfloat16, true>(a, dev.sm_count, st); break;
    default: s = grad_t<__half, true>(a, dev.sm_count, st); break;
  }
  if (scales) cudaFreeAsync(scales, st);
  return s;
}

}  // namespace fxtx
