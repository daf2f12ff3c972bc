// few.cu — float32 results of few rows on the CUDA cores: out = act(X W + b) + R for up to 16 rows
// (weights stored by rows) or 8 (by columns).
//
// Bound: HBM, the weights' stream (2 m operations for each entry of W: with 16 rows about 70 % of
// the fp32 pipe). W is read once, where it lies, whatever its order, pitch and alignment; on the
// tensor cores it is first split into three planes, four times the traffic. 4096 x 4096: one row 18 us
// by rows and 14 us by columns (49 us on the tensor cores), 8 rows 25 and 38 us, 16 rows 29 us by rows (49);
// by columns 16 rows took 141 us (50), since its lanes need all of X's rows for every feature. One row of
// 8192 x 8192: 46 us (5.8 TB/s). bfloat16 and float16 have no planes to make and stay on the tensor cores: 8.1 us
// for one row of 4096 x 4096.
//
// A cluster of R CTAs takes one block of columns, each CTA a part of the features; X's rows sit in
// shared memory. W stored by rows: a lane takes 4 neighbouring columns of 4 features at a time, so
// that a row of X gives 4 factors in one read; LC lanes lie along the columns, 32, or 8 where the
// columns are too few to give every SM a block. W stored by columns: a lane takes 4 neighbouring features
// of 4 columns, and a warp adds its lanes. The CTAs' sums go to the CTA that finishes each of them
// (distributed shared memory) and are added in order: one launch, no workspace, the same bits on
// every call. Unaligned weights are read entry by entry, neighbouring lanes still reading neighbouring
// entries.
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "kernels.h"
#include "linear.h"
#include "product.cuh"
#include "tc.cuh"

namespace fxtx {
namespace {

constexpr int THREADS = 256, WARPS = 8;
constexpr int SLICE = 1024;  // features of X held at a time
constexpr int CC = 4;        // columns a warp takes of weights stored by columns

constexpr int VE = 4;        // entries of W a lane takes in one read

struct FewArgs {
  int64_t m;
  int n, k;  // features (the sums' length), columns of the result
  const void* X;
  int64_t ldx, x_planes;  // x_planes > 0: X as its three bfloat16 planes
  const float* W;
  int64_t ld;
  Epilogue e;
  int R;        // CTAs a cluster
  int64_t per;  // features a CTA
  bool wide;   // W's rows (columns) are 16-byte aligned
};

__device__ __forceinline__ float x_at(const FewArgs& a, int64_t i, int64_t j) {
  if (a.x_planes == 0) return static_cast<const float*>(a.X)[i * a.ldx + j];
  const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.X) + i * a.ldx + j;
  return to_f32(p[0]) + (to_f32(p[a.x_planes]) + to_f32(p[2 * a.x_planes]));  // exact
}

// VE entries from p on (`step` apart where they are read one by one), those before `left` only.
__device__ __forceinline__ void load_vec(const float* p, int step, int left, bool wide, float (&x)[VE]) {
  if (wide && left >= VE) {
    const float4 v = __ldcs(reinterpret_cast<const float4*>(p));
    x[0] = v.x; x[1] = v.y; x[2] = v.z; x[3] = v.w;
  } else {
#pragma unroll
    for (int i = 0; i < VE; ++i) x[i] = i * step < left ? p[i * step] : 0.f;
  }
}

// LC: lanes along the columns of weights stored by rows; 0: stored by columns.
template <int MR, int LC>
struct Shape {
  static constexpr int COLS = LC == 0 ? WARPS * CC : LC * VE;  // columns a CTA takes
  static constexpr int OUT = MR * COLS;
  // X's slice, then the warps' sums
  static constexpr int XS = LC != 0 && WARPS * OUT > MR * SLICE ? WARPS * OUT : MR * SLICE;
  static constexpr size_t BYTES = (size_t)(XS + OUT) * 4;
};

template <int MR, int LC>
__global__ void __launch_bounds__(THREADS) few_kernel(const __grid_constant__ FewArgs a) {
  using S = Shape<MR, LC>;
  constexpr int COLS = S::COLS, OUT = S::OUT;
  extern __shared__ __align__(16) float smem[];
  float *xs = smem, *red = smem + S::XS;  // [MR][SLICE], then [WARPS][OUT]; [from][OUT / R]
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int R = a.R, rank = R > 1 ? (int)cluster_rank() : 0;
  const int c0 = (int)(blockIdx.x / (unsigned)R) * COLS;
  const int64_t i0 = (int64_t)blockIdx.y * MR;
  // (64 bits: the last CTA's range, rounded up, and the slice after the last may begin beyond 2^31)
  const int64_t j_begin = rank * a.per, j_end = min((int64_t)a.n, j_begin + a.per);
  const float* W = a.W;
  if (R > 1) cluster_arrive();  // waited for before the first store to another CTA
  after_previous();

  constexpr int AX = LC == 0 ? CC : VE;
  float acc[MR][AX] = {};
  for (int64_t j0 = j_begin; j0 < j_end; j0 += SLICE) {
    const int len = (int)min((int64_t)SLICE, j_end - j0);
    __syncthreads();
    // up to a whole step of the lanes; what lies beyond the features is zero
    const int padded = (len + 32 * VE - 1) / (32 * VE) * (32 * VE);
    for (int j = tid; j < padded; j += THREADS) {
      float x[MR];
#pragma unroll
      for (int i = 0; i < MR; ++i) x[i] = j < len && i0 + i < a.m ? x_at(a, i0 + i, j0 + j) : 0.f;
#pragma unroll
      for (int i = 0; i < MR; ++i) xs[i * SLICE + j] = x[i];
    }
    __syncthreads();
    if constexpr (LC != 0) {
      constexpr int G = 32 / LC;  // groups of 4 features a warp takes
      const int x = lane % LC, c = c0 + (a.wide ? x * VE : x), step = a.wide ? 1 : LC;
#pragma unroll 2
      for (int j = (warp * G + lane / LC) * 4; j < len; j += WARPS * G * 4) {
        float w[4][VE];
#pragma unroll
        for (int s = 0; s < 4; ++s)
          load_vec(W + (j0 + j + s) * a.ld + c, step, j + s < len ? a.k - c : 0, a.wide, w[s]);
#pragma unroll
        for (int i = 0; i < MR; ++i) {
          const float4 y = *reinterpret_cast<const float4*>(xs + i * SLICE + j);
#pragma unroll
          for (int q = 0; q < VE; ++q)
            acc[i][q] = fmaf(y.w, w[3][q], fmaf(y.z, w[2][q], fmaf(y.y, w[1][q], fmaf(y.x, w[0][q], acc[i][q]))));
        }
      }
    } else {
      const int c = c0 + warp * CC;
#pragma unroll 2
      for (int j = a.wide ? lane * VE : 0; j < len; j += 32 * VE) {
        // feature q of the lane: neighbours (wide), or 32 apart
        const int jj = a.wide ? j : j + lane, step = a.wide ? 1 : 32;
        float w[CC][VE];
#pragma unroll
        for (int s = 0; s < CC; ++s)
          load_vec(W + (int64_t)(c + s) * a.ld + j0 + jj, step, c + s < a.k ? len - jj : 0, a.wide, w[s]);
#pragma unroll
        for (int i = 0; i < MR; ++i) {
          float x[VE];
          if (a.wide) {
            *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(xs + i * SLICE + jj);
          } else {
#pragma unroll
            for (int q = 0; q < VE; ++q) x[q] = xs[i * SLICE + jj + 32 * q];
          }
#pragma unroll
          for (int s = 0; s < CC; ++s)
#pragma unroll
            for (int q = 0; q < VE; ++q) acc[i][s] = fmaf(x[q], w[s][q], acc[i][s]);
        }
      }
    }
  }

  // each sum of the CTA to the CTA that finishes it
  __syncthreads();
  if (R > 1) cluster_wait();
  const int share = OUT / R;
  auto send = [&](int o, float v) {
    const int to = o / share, at = rank * share + o % share;
    if (R > 1) st_cluster(cluster_addr(red, (uint32_t)to) + 4u * (uint32_t)at, v);
    else red[at] = v;
  };
  if constexpr (LC != 0) {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int q = 0; q < VE; ++q) {
        float v = acc[i][q];
#pragma unroll
        for (int o = LC; o < 32; o *= 2) v += shfl_xor(v, o);
        if (lane < LC) xs[warp * OUT + i * COLS + (a.wide ? lane * VE + q : lane + LC * q)] = v;
      }
    __syncthreads();
    for (int o = tid; o < OUT; o += THREADS) {
      float v = 0.f;
#pragma unroll
      for (int w = 0; w < WARPS; ++w) v += xs[w * OUT + o];
      send(o, v);
    }
  } else {
#pragma unroll
    for (int i = 0; i < MR; ++i)
#pragma unroll
      for (int s = 0; s < CC; ++s) {
        const float v = group_sum<32>(acc[i][s]);
        if (lane == (i * CC + s) % 32) send(i * COLS + warp * CC + s, v);
      }
  }
  __syncthreads();
  if (R > 1) cluster_sync();
  const Finish<float> fin(a.e, a.m, a.k);
  for (int o = tid; o < share; o += THREADS) {
    float v = 0.f;
    for (int s = 0; s < R; ++s) v += red[s * share + o];
    const int at = rank * share + o;
    fin.one(i0 + at / COLS, c0 + at % COLS, v);
  }
}

template <int MR, int LC>
cudaError_t launch(FewArgs a, int sm_count, cudaStream_t st) {
  using S = Shape<MR, LC>;
  const int64_t blocks = (a.k + S::COLS - 1) / S::COLS, chunks = (a.m + MR - 1) / MR;
  // CTAs enough for two a SM, each with 64 features at least
  a.R = 1;
  while (a.R < 8 && blocks * chunks * a.R < 2 * sm_count && a.n >= 128 * a.R) a.R *= 2;
  a.per = (((int64_t)a.n + a.R - 1) / a.R + 31) / 32 * 32;
  const void* k = (const void*)few_kernel<MR, LC>;
  cudaError_t e = ensure_smem(k, S::BYTES);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(blocks * a.R), (unsigned)chunks);
  cfg.blockDim = dim3(THREADS);
  cfg.dynamicSmemBytes = S::BYTES;
  cfg.stream = st;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;  // (see after_previous)
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)a.R;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = a.R > 1 ? 2 : 1;
  void* args[] = {&a};
  return cudaLaunchKernelExC(&cfg, k, args);
}

template <int LC>
cudaError_t launch_rows(const FewArgs& a, int sm_count, cudaStream_t st) {
  if (a.m <= 1) return launch<1, LC>(a, sm_count, st);
  if (a.m <= 2) return launch<2, LC>(a, sm_count, st);
  if (a.m <= 4) return launch<4, LC>(a, sm_count, st);
  if constexpr (LC != 0) {
    if (a.m > 8) return launch<16, LC>(a, sm_count, st);
  }
  return launch<8, LC>(a, sm_count, st);
}

}  // namespace

fxtx_status_t run_few(int64_t m, int64_t n, int64_t k, const void* X, int64_t ldx, int64_t x_planes, const float* W,
                      int64_t ld, bool by_column, const Epilogue& e, const DeviceInfo& dev, cudaStream_t st) {
  FewArgs a = {};
  a.m = m;
  a.n = (int)n;
  a.k = (int)k;
  a.X = X;
  a.ldx = ldx;
  a.x_planes = x_planes;
  a.W = W;
  a.ld = ld;
  a.e = e;
  a.wide = ((uintptr_t)W & 15u) == 0 && ld % 4 == 0;
  const bool narrow = (k + 127) / 128 * 8 < dev.sm_count;
  const cudaError_t err = by_column ? launch_rows<0>(a, dev.sm_count, st)
                          : narrow  ? launch_rows<8>(a, dev.sm_count, st)
                                    : launch_rows<32>(a, dev.sm_count, st);
  if (err == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

}  // namespace fxtx
