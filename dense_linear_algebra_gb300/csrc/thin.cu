// thin.cu — the linear layer and its gradient for at most 64 features and 64 outputs: every
// entry of X, G, Z, R is read once, by the thread that uses it, and a row's results are
// written in one piece.
//
// Bound: HBM. Such layers do n k / (n + k) multiply-adds for each value moved, too few to pay
// for the way through shared and tensor memory: on the tcgen05 kernels a 64-wide stage of kk and
// a 64-wide tile are half empty, and their eight epilogue warps a SM are what they wait for
// (1,000,000 x 32, 32 outputs: 109 us in bfloat16, 201 us in float32 with its three planes; here 26 and 68 us,
// the latter 5.6 TB/s, and their gradients 88 and 99 us, held back by the latency of few warps). Here
// a warp forms 16 rows with m16n8k16 products on registers, warps are independent of one another,
// and the next rows' loads are in flight meanwhile.
//
// Which column sits in which fragment register is free, as long as both operands agree: of
// a row of 16 KS entries, lane t of a quad takes the 4 KS neighbouring ones from 4 KS t on (one
// to four 16-byte loads), and of a row of 8 NT results the 2 NT from 2 NT t on. W is laid out to match
// once a CTA, in shared memory.
//
// dW = X^T D takes both operands transposed: movmatrix turns the 8 x 8 blocks that dX = D W^T
// already has in registers. A warp keeps its dW and db over all of its rows; a CTA's warps
// are added in order into a workspace and a second kernel adds the CTAs, so both come out the same
// on every call.
//
// float32: each value is split into three bfloat16 terms (exactly) and six products are formed
// (the rest is at most 2^-26 of a term); sums over rows leave the tensor cores after each 16 rows and
// are added in fp32 registers. D stays in fp32 but for that split; of 16-bit types it is rounded
// to the type, as the products take it.
//
// 16 bits: a warp's dW stays in the products' accumulators, which cut off 1e-7 of a sum of terms of one sign every
// 16 rows. From 8,192 rows a warp on (20,000,000 in all) more CTAs than fit are launched instead, so
// that 5e-5 is left at most, a tenth of float16's rounding; 200,000,000 rows on a grid that fits were 5.1e-4 off.
#include "thin.cuh"

namespace fxtx {
namespace {

template <typename T, int KS, int NT>
__global__ void __launch_bounds__(THREADS) thin_kernel(const ThinArgs a) {
  __shared__ uint2 ws[KS * NT * Term<T>::P * 32];
  after_previous();
  stage_operand<T, KS, NT>(ws, static_cast<const T*>(a.W), a.ws0, a.ws1, a.n, a.k);
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int64_t tiles = (a.m + 15) / 16, step = (int64_t)gridDim.x * WARPS;
  const Rows<T, KS> rows(a.X, a.ldx, a.n);
  const Finish<T> fin(a.e, a.m, a.k);
  int64_t w = (int64_t)blockIdx.x * WARPS + (threadIdx.x >> 5);
  Chunk<T, KS> next;
  rows.load(w * 16, a.m, next);
  __syncthreads();
  for (; w < tiles; w += step) {
    const Chunk<T, KS> x = next;
    float c[2][2 * NT];
    rows.load((w + step) * 16, a.m, next);
    rows_times<T, KS, NT>(x, ws, c);
#pragma unroll
    for (int h = 0; h < 2; ++h) fin.template row<2 * NT>(w * 16 + g + 8 * h, 2 * NT * t, c[h]);
  }
}

template <typename T, int KS, int NT>
cudaError_t launch_layer(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return launch_kernel(thin_kernel<T, KS, NT>, dim3(grid_of<thin_kernel<T, KS, NT>>(a.m, sm_count)), THREADS, 0, st, a);
}

template <typename T, int KS>
cudaError_t layer_k(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return a.k <= 16 ? launch_layer<T, KS, 2>(a, sm_count, st)
                   : a.k <= 32 ? launch_layer<T, KS, 4>(a, sm_count, st) : launch_layer<T, KS, 8>(a, sm_count, st);
}
template <typename T>
cudaError_t layer_t(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return a.n <= 16 ? layer_k<T, 1>(a, sm_count, st)
                   : a.n <= 32 ? layer_k<T, 2>(a, sm_count, st) : layer_k<T, 4>(a, sm_count, st);
}

}  // namespace

bool thin_shape(int64_t n, int64_t k) { return n >= 1 && n <= kThin && k >= 1 && k <= kThin; }

fxtx_status_t run_thin_linear(const LayerArgs& l, const DeviceInfo& dev, cudaStream_t st) {
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
  cudaError_t e;
  switch (l.type) {
    case FXTX_F32: e = layer_t<float>(a, dev.sm_count, st); break;
    case FXTX_BF16: e = layer_t<__nv_bfloat16>(a, dev.sm_count, st); break;
    default: e = layer_t<__half>(a, dev.sm_count, st); break;
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

fxtx_status_t run_thin_grad(const LayerArgs& l, const GradArgs& g, const DeviceInfo& dev, cudaStream_t st) {
  ThinArgs a = {};
  a.m = l.m;
  a.n = (int)l.n;
  a.k = (int)l.k;
  a.X = l.X;
  a.ldx = l.ldx;
  a.W = l.W;
  a.ws0 = l.w_trans ? 1 : l.ldw;
  a.ws1 = l.w_trans ? l.ldw : 1;
  a.G = g.G;
  a.ldg = g.ldg;
  a.Z = g.Z;
  a.ldz = g.ldz;
  a.act = g.act;
  a.DX = g.DX;
  a.lddx = g.lddx;
  a.DW = g.DW;
  a.dws0 = l.w_trans ? 1 : g.lddw;
  a.dws1 = l.w_trans ? g.lddw : 1;
  a.DB = g.DB;
  switch (l.type) {
    case FXTX_F32: return grad_t<float, false>(a, dev.sm_count, st);
    case FXTX_BF16: return grad_t<__nv_bfloat16, false>(a, dev.sm_count, st);
    default: return grad_t<__half, false>(a, dev.sm_count, st);
  }
}

}  // namespace fxtx
