// thin_loss_f32.cu — softmax cross entropy of many float32 rows on at most 16 classes (the gradient 12) and 64 features, and its
// gradient, on the CUDA cores: plain fp32 multiply-adds, two an instruction.
//
// Bound: HBM (X read once) and the multiply-adds, n k a row for z and as many for dW (1,000,000 x 32, 10 classes: 21 us and 17 us).
// On the tensor cores float32 takes six products of bfloat16 terms, and half of a fragment is padding at 10 classes: that
// form of the gradient takes 60 us.
//
// A warp takes tiles of 64 rows, which come by asynchronous copies into shared memory (while the other warps work: a second
// buffer would leave 10 warps a SM), with a pitch that keeps both ways of reading free of bank conflicts: a lane two rows for z,
// the softmax and D; then a lane two features for dW, whose sums stay in its registers, the rows shared out among the
// lanes that are left. D goes through shared memory in between. What it waits for is shared memory: with a row a lane W is
// read twice as often (52 us, two rows 48). The warps' sums are added in turn, the CTAs' by a second kernel in order.
#include <algorithm>

#include "act.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "loss.h"

namespace fxtx {
namespace {

constexpr int MOST_CLASSES = 16, MOST_GRAD_CLASSES = 12;

struct TallArgs {
  int64_t m;
  int n, k;
  const float* X;
  int64_t ldx;
  const float* W;
  int64_t ws0, ws1;  // entry (j, c) of W at W[j * ws0 + c * ws1]
  const float* b;
  bool wide;         // rows of whole 16 bytes, aligned
  LossArgs q;
  bool wide_dx;
  int64_t dws0, dws1;
  float* part;       // [CTA][features + 1][pitch of the classes] sums of dW and, last, db
};

using f2 = unsigned long long;
__device__ __forceinline__ f2 pack2(float x, float y) {
  f2 r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(x), "f"(y));
  return r;
}
__device__ __forceinline__ float2 unpack2(f2 v) {
  float2 r;
  asm("mov.b64 {%0, %1}, %2;" : "=f"(r.x), "=f"(r.y) : "l"(v));
  return r;
}
__device__ __forceinline__ f2 add2(f2 a, f2 b) {
  f2 r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// `bytes` (4 or 16) from src, or as many zeros.
template <int BYTES>
__device__ __forceinline__ void copy_async(float* dst, const float* src, bool there) {
  if constexpr (BYTES == 16)
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 16 : 0) : "memory");
  else
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(smem_addr(dst)), "l"(src), "r"(there ? 4 : 0) : "memory");
}

// N: features, padded; KP: pairs of classes. R: rows a lane has.
template <int N, int KP>
struct Tall {
  static constexpr int R = 2, ROWS = 32 * R, PITCH = N + 4;
  static constexpr int DP = (2 * KP + 3) / 4 * 4;           // pitch of D and of W
  static constexpr int FL = N / 2, RS = 32 / FL;            // lanes a row takes for dW, and rows side by side
  static constexpr int TILE = ROWS * PITCH, WARP = TILE + ROWS * DP;  // floats: a tile, a warp's
  static constexpr int FIXED = (N + 1) * DP;                // W and the biases
  static constexpr int WARPS = std::min(16, (int)((220 * 1024 / 4 - FIXED) / WARP));
  static constexpr size_t BYTES = (size_t)(FIXED + WARPS * WARP) * 4;
  static_assert(WARP >= FIXED, "room for the warps' sums at the end");
};

// KP pairs from p on (16-byte aligned).
template <int KP>
__device__ __forceinline__ void load_pairs(const float* p, f2 (&x)[KP]) {
#pragma unroll
  for (int i = 0; i + 1 < KP; i += 2) {
    const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(p + 2 * i);
    x[i] = v.x;
    x[i + 1] = v.y;
  }
  if constexpr (KP % 2) x[KP - 1] = *reinterpret_cast<const f2*>(p + 2 * (KP - 1));
}

// MODE 0: the loss; 1: dW and db; 2: dX too.
template <int N, int KP, int MODE>
__global__ void __launch_bounds__((Tall<N, KP>::WARPS * 32), 1) tall_loss_kernel(const __grid_constant__ TallArgs a) {
  using C = Tall<N, KP>;
  constexpr int R = C::R, DP = C::DP, PITCH = C::PITCH;
  extern __shared__ __align__(16) float smem[];
  float *Ws = smem, *bias = smem + N * DP;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  float *tiles = smem + C::FIXED + warp * C::WARP, *ds = tiles + C::TILE;
  after_previous();
  for (int i = threadIdx.x; i < N * DP; i += C::WARPS * 32) {
    const int j = i / DP, c = i % DP;
    Ws[i] = j < a.n && c < a.k ? a.W[j * a.ws0 + c * a.ws1] : 0.f;
  }
  for (int c = threadIdx.x; c < DP; c += C::WARPS * 32) bias[c] = c >= a.k ? -INFINITY : a.b ? a.b[c] : 0.f;
  const int64_t count = (a.m + C::ROWS - 1) / C::ROWS, step = (int64_t)gridDim.x * C::WARPS;
  int64_t tile = (int64_t)blockIdx.x * C::WARPS + warp;

  auto fetch = [&](int64_t i, float* to) {
    if (i < count) {
      const float* X = a.X + i * C::ROWS * a.ldx;
      const int rows = (int)min((int64_t)C::ROWS, a.m - i * C::ROWS);
      if (a.wide) {
#pragma unroll 4
        for (int e = lane; e < C::ROWS * (N / 4); e += 32) {
          const int r = e / (N / 4), c = e % (N / 4) * 4;
          const bool there = r < rows && c < a.n;
          copy_async<16>(to + r * PITCH + c, there ? X + r * a.ldx + c : a.X, there);
        }
      } else {
#pragma unroll 4
        for (int e = lane; e < C::ROWS * N; e += 32) {
          const int r = e / N, c = e % N;
          const bool there = r < rows && c < a.n;
          copy_async<4>(to + r * PITCH + c, there ? X + r * a.ldx + c : a.X, there);
        }
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  // a row's label, lse and weight, a tile ahead
  int64_t label_n[R];  // as they come
  float lse_n[R], g_n[R];
  auto fetch_rows = [&](int64_t i) {
#pragma unroll
    for (int y = 0; y < R; ++y) {
      const int64_t r = i * C::ROWS + lane + 32 * y;
      const bool in = r < a.m;
      label_n[y] = !in ? -1 : a.q.labels64 ? static_cast<const int64_t*>(a.q.labels)[r] : (int64_t)static_cast<const int32_t*>(a.q.labels)[r];
      lse_n[y] = MODE > 0 && in ? a.q.lse_in[r] : 0.f;
      g_n[y] = MODE > 0 && in && a.q.g ? a.q.g[r] : 1.f;
    }
  };
  fetch(tile, tiles);
  fetch_rows(tile);
  __syncthreads();

  f2 dw[MODE ? 2 : 1][MODE ? KP : 1] = {}, db[MODE ? KP : 1] = {};
  for (; tile < count; tile += step) {
    float* x = tiles;
    int label[R];
    float lse[R], g[R];
#pragma unroll
    for (int y = 0; y < R; ++y) {
      label[y] = label_n[y] < 0 || label_n[y] >= a.k ? -1 : (int)label_n[y];
      lse[y] = lse_n[y];
      g[y] = label[y] >= 0 ? a.q.gain * g_n[y] : 0.f;
    }
    fetch_rows(tile + step);
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncwarp();
    // z of the lane's rows
    f2 z[R][KP];
    {
      f2 b[KP];
      load_pairs<KP>(bias, b);
#pragma unroll
      for (int y = 0; y < R; ++y)
#pragma unroll
        for (int c = 0; c < KP; ++c) z[y][c] = 0;
#pragma unroll 2
      for (int j = 0; j < N; j += 4) {
        float4 v[R];
#pragma unroll
        for (int y = 0; y < R; ++y) v[y] = *reinterpret_cast<const float4*>(x + (lane + 32 * y) * PITCH + j);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f2 w[KP];
          load_pairs<KP>(Ws + (j + q) * DP, w);
#pragma unroll
          for (int y = 0; y < R; ++y) {
            const float s = q == 0 ? v[y].x : q == 1 ? v[y].y : q == 2 ? v[y].z : v[y].w;
            const f2 ss = pack2(s, s);
#pragma unroll
            for (int c = 0; c < KP; ++c) z[y][c] = fma2(ss, w[c], z[y][c]);
          }
        }
      }
#pragma unroll
      for (int y = 0; y < R; ++y)
#pragma unroll
        for (int c = 0; c < KP; ++c) z[y][c] = add2(z[y][c], b[c]);
    }
    if constexpr (MODE == 0) {
      __syncwarp();
      fetch(tile + step, tiles);
#pragma unroll
      for (int y = 0; y < R; ++y) {
        const int64_t r = tile * C::ROWS + lane + 32 * y;
        float top = -INFINITY, target = 0.f, sum = 0.f;
#pragma unroll
        for (int c = 0; c < KP; ++c) {
          const float2 v = unpack2(z[y][c]);
          top = fmaxf(top, fmaxf(v.x, v.y));
          target += (2 * c == label[y] ? v.x : 0.f) + (2 * c + 1 == label[y] ? v.y : 0.f);
        }
        const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
        for (int c = 0; c < KP; ++c) {
          const float2 v = unpack2(z[y][c]);
          sum += expf(v.x - from) + expf(v.y - from);
        }
        const float rest = logf(sum);
        if (r >= a.m) continue;
        if (a.q.loss) a.q.loss[r] = label[y] >= 0 ? (from - target) + rest : 0.f;
        if (a.q.lse) a.q.lse[r] = from + rest;
      }
      continue;
    }
    // D, to shared memory too
#pragma unroll
    for (int y = 0; y < R; ++y) {
      const bool on = label[y] >= 0;
      float* d = ds + (lane + 32 * y) * DP;
#pragma unroll
      for (int c = 0; c < KP; ++c) {
        float2 v = unpack2(z[y][c]);
        v.x = on ? g[y] * expf(v.x - lse[y]) : 0.f;
        v.y = on ? g[y] * expf(v.y - lse[y]) : 0.f;
        v.x -= 2 * c == label[y] ? g[y] : 0.f;
        v.y -= 2 * c + 1 == label[y] ? g[y] : 0.f;
        z[y][c] = pack2(v.x, v.y);
        db[MODE ? c : 0] = add2(db[MODE ? c : 0], z[y][c]);
        *reinterpret_cast<f2*>(d + 2 * c) = z[y][c];
      }
    }
    __syncwarp();
    if (a.q.DW) {
      const float *xf = x + 2 * (lane % C::FL), *xr = xf + lane / C::FL * PITCH, *dr = ds + lane / C::FL * DP;
#pragma unroll 4
      for (int r = 0; r < C::ROWS; r += C::RS) {
        const float2 v = *reinterpret_cast<const float2*>(xr + r * PITCH);
        f2 d[KP];
        load_pairs<KP>(dr + r * DP, d);
        const f2 v0 = pack2(v.x, v.x), v1 = pack2(v.y, v.y);
#pragma unroll
        for (int c = 0; c < KP; ++c) {
          dw[0][MODE ? c : 0] = fma2(v0, d[c], dw[0][MODE ? c : 0]);
          dw[MODE ? 1 : 0][MODE ? c : 0] = fma2(v1, d[c], dw[MODE ? 1 : 0][MODE ? c : 0]);
        }
      }
    }
    __syncwarp();
    if constexpr (MODE == 2) {
      // dX over the tile, a lane a row, and from there to memory in whole lines
#pragma unroll 1
      for (int j = 0; j < N; j += 4) {
        float o[R][4];
#pragma unroll
        for (int q = 0; q < 4; ++q) {
          f2 w[KP];
          load_pairs<KP>(Ws + (j + q) * DP, w);
#pragma unroll
          for (int y = 0; y < R; ++y) {
            f2 s = 0;
#pragma unroll
            for (int c = 0; c < KP; ++c) s = fma2(z[y][c], w[c], s);
            o[y][q] = unpack2(s).x + unpack2(s).y;
          }
        }
#pragma unroll
        for (int y = 0; y < R; ++y)
          *reinterpret_cast<float4*>(x + (lane + 32 * y) * PITCH + j) = make_float4(o[y][0], o[y][1], o[y][2], o[y][3]);
      }
      __syncwarp();
      float* DX = static_cast<float*>(a.q.DX) + tile * C::ROWS * a.q.lddx;
      const int rows = (int)min((int64_t)C::ROWS, a.m - tile * C::ROWS);
      if (a.wide_dx) {
#pragma unroll 4
        for (int e = lane; e < C::ROWS * (N / 4); e += 32) {
          const int r = e / (N / 4), c = e % (N / 4) * 4;
          if (r < rows && c < a.n) *reinterpret_cast<float4*>(DX + r * a.q.lddx + c) = *reinterpret_cast<const float4*>(x + r * PITCH + c);
        }
      } else {
#pragma unroll 4
        for (int e = lane; e < C::ROWS * N; e += 32) {
          const int r = e / N, c = e % N;
          if (r < rows && c < a.n) DX[r * a.q.lddx + c] = x[r * PITCH + c];
        }
      }
      __syncwarp();
    }
    fetch(tile + step, tiles);
  }
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  if constexpr (MODE == 0) return;
  if (!a.part) return;

  // the sums: over the lanes that share features, over the warps in order
  __syncthreads();
  float* sums = smem + C::FIXED;  // [warp][N + 1][DP], over the tiles
  float v[2][2 * KP], s[2 * KP];
#pragma unroll
  for (int c = 0; c < KP; ++c) {
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      v[f][2 * c] = unpack2(dw[MODE ? f : 0][MODE ? c : 0]).x;
      v[f][2 * c + 1] = unpack2(dw[MODE ? f : 0][MODE ? c : 0]).y;
    }
    s[2 * c] = unpack2(db[MODE ? c : 0]).x;
    s[2 * c + 1] = unpack2(db[MODE ? c : 0]).y;
  }
#pragma unroll
  for (int c = 0; c < 2 * KP; ++c) {
#pragma unroll
    for (int o = C::FL; o < 32; o <<= 1) {
      v[0][c] += shfl_xor(v[0][c], o);
      v[1][c] += shfl_xor(v[1][c], o);
    }
    s[c] = group_sum<32>(s[c]);
  }
  float* own = sums + warp * C::FIXED;
  if (lane < C::FL)
#pragma unroll
    for (int c = 0; c < 2 * KP; ++c) {
      own[2 * lane * DP + c] = v[0][c];
      own[(2 * lane + 1) * DP + c] = v[1][c];
      if (lane == 0) own[N * DP + c] = s[c];
    }
  __syncthreads();
  for (int i = threadIdx.x; i < C::FIXED; i += C::WARPS * 32) {
    float t = 0.f;
#pragma unroll 4
    for (int w = 0; w < C::WARPS; ++w) t += sums[w * C::FIXED + i];
    a.part[(int64_t)blockIdx.x * C::FIXED + i] = t;
  }
}

// dW and db from the CTAs' sums, in order: 8 entries a CTA, a warp each.
__global__ void __launch_bounds__(256) tall_join_kernel(const __grid_constant__ TallArgs a, int N, int DP, int parts) {
  const int lane = threadIdx.x & 31, e = (int)(blockIdx.x * 8 + (threadIdx.x >> 5)), j = e / DP, c = e % DP;
  after_previous();
  if (j > N || c >= a.k || (j >= a.n && j != N)) return;
  const int size = (N + 1) * DP;
  float s = 0.f;
#pragma unroll 8
  for (int p = lane; p < parts; p += 32) s += a.part[(int64_t)p * size + e];
  s = group_sum<32>(s);
  if (lane != 0) return;
  if (j < N) {
    if (a.q.DW) static_cast<float*>(a.q.DW)[j * a.dws0 + c * a.dws1] = s;
  } else if (a.q.DB) {
    static_cast<float*>(a.q.DB)[c] = s;
  }
}

template <int N, int KP, int MODE>
fxtx_status_t launch(TallArgs a, const DeviceInfo& dev, cudaStream_t st) {
  using C = Tall<N, KP>;
  cudaError_t e = ensure_smem((const void*)tall_loss_kernel<N, KP, MODE>, C::BYTES);
  const int64_t tiles = (a.m + C::ROWS - 1) / C::ROWS, grid = std::min<int64_t>((tiles + C::WARPS - 1) / C::WARPS, dev.sm_count);
  if (MODE > 0 && (a.q.DW || a.q.DB) && e == cudaSuccess) {
    const fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)grid * C::FIXED * 4, st);
    if (s != FXTX_OK) return s;
  }
  if (e == cudaSuccess) e = launch_kernel(tall_loss_kernel<N, KP, MODE>, dim3((unsigned)grid), C::WARPS * 32, C::BYTES, st, a);
  if (a.part) {
    if (e == cudaSuccess) e = launch_kernel(tall_join_kernel, dim3((unsigned)((C::FIXED + 7) / 8)), 256, 0, st, a, N, C::DP, (int)grid);
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}
template <int N, int KP>
fxtx_status_t launch_mode(const TallArgs& a, int mode, const DeviceInfo& dev, cudaStream_t st) {
  if constexpr (2 * KP <= MOST_GRAD_CLASSES) {
    if (mode > 0) return mode == 1 ? launch<N, KP, 1>(a, dev, st) : launch<N, KP, 2>(a, dev, st);
  }
  return launch<N, KP, 0>(a, dev, st);
}
// Pairs of classes as many as there are (padded to the next even number of pairs, the gradient of 1,000,000 x 32 takes 44 us for 6
// classes, as they are 37; its loss 40 for 14 classes, as they are 37).
template <int N, int KP = 1>
fxtx_status_t launch_classes(const TallArgs& a, int mode, const DeviceInfo& dev, cudaStream_t st) {
  if constexpr (KP < MOST_CLASSES / 2) {
    if (a.k > 2 * KP) return launch_classes<N, KP + 1>(a, mode, dev, st);
  }
  return launch_mode<N, KP>(a, mode, dev, st);
}

fxtx_status_t run(const LayerArgs& l, const LossArgs& q, int mode, const DeviceInfo& dev, cudaStream_t st) {
  TallArgs a = {};
  a.m = l.m;
  a.n = (int)l.n;
  a.k = (int)l.k;
  a.X = static_cast<const float*>(l.X);
  a.ldx = l.ldx;
  a.W = static_cast<const float*>(l.W);
  a.ws0 = l.w_trans ? 1 : l.ldw;
  a.ws1 = l.w_trans ? l.ldw : 1;
  a.b = static_cast<const float*>(l.e.bias);
  a.wide = ((uintptr_t)l.X & 15u) == 0 && l.ldx % 4 == 0 && l.n % 4 == 0;
  a.q = q;
  a.wide_dx = ((uintptr_t)q.DX & 15u) == 0 && q.lddx % 4 == 0 && l.n % 4 == 0;
  a.dws0 = l.w_trans ? 1 : q.lddw;
  a.dws1 = l.w_trans ? q.lddw : 1;
  return l.n <= 16 ? launch_classes<16>(a, mode, dev, st) : l.n <= 32 ? launch_classes<32>(a, mode, dev, st) : launch_classes<64>(a, mode, dev, st);
}

}  // namespace

// Where this way is the faster one (us, here and on the tensor cores, of the loss / dW and db / dX too):
//   1,000,000 x 32   6 classes 26 / 37 / 59 and 41 / 60 / 92, 12 classes 32 / 53 / 81 and 41 / 60 / 92, 14 classes 37 / 72 / 116, 16
//                    classes 40 / 91 / 136; x 24, 13 classes 35 / 68 / 112 and 47 / 80 / 109
//   500,000 x 64     8 classes 30 / 47 / 75 and 33 / 56 / 91, 10 classes 34 / 57 / 90, 12 classes 37 / 61 / 98 and 33 / 56 / 91
//   rows of 32       2 classes, 20,000 rows 4.2 / 6.7 / 9.5 and 3.8 / 8.8 / 9.8; 10 classes, 20,000 6.0 / 10.7 / 14.7 and 4.1 / 9.2 / 9.7,
//                    50,000 6.0 / 11.2 / 15.3 and 4.9 / 11.9 / 13.1, 100,000 6.0 / 12.0 / 16.1 and 7.0 / 14.0 / 16.1 (a warp takes 64
//                    rows at a time: few rows leave SMs without, for longer the more classes there are)
bool tall_loss_shape(const LayerArgs& l, bool grad) {
  return l.type == FXTX_F32 && l.n <= 64 && l.k <= (grad ? MOST_GRAD_CLASSES : MOST_CLASSES) && l.n * l.k <= 512 &&
         l.m >= (grad ? 5000 : 8000) * l.k;
}
fxtx_status_t run_tall_loss(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st) { return run(l, a, 0, dev, st); }
fxtx_status_t run_tall_loss_grad(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  return run(l, a, a.DX ? 2 : 1, dev, st);
}

}  // namespace fxtx
