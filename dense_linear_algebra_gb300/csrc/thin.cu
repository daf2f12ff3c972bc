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
#include <algorithm>
#include <type_traits>

#include "act.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "linear.h"
#include "product.cuh"

namespace fxtx {
namespace {

constexpr int THREADS = 128, WARPS = THREADS / 32;
constexpr int64_t MOST = 512;  // times 16 rows that a warp adds to its 16-bit dW

struct ThinArgs {
  int64_t m;
  int n, k;
  const void* X;
  int64_t ldx;
  const void* W;
  int64_t ws0, ws1;  // entry (j, c) of W at W[j * ws0 + c * ws1]
  Epilogue e;        // the layer's
  // the gradient's
  const void* G;
  int64_t ldg;
  const void* Z;
  int64_t ldz;
  int act;
  void* DX;
  int64_t lddx;
  void* DW;
  int64_t dws0, dws1;
  void* DB;
  float* part;  // the CTAs' sums of dW and db, as their lanes hold them
};

template <typename T>
struct Term {  // the type of the products' operands, and how many terms a value takes
  using type = T;
  static constexpr int P = 1;
};
template <>
struct Term<float> {
  using type = __nv_bfloat16;
  static constexpr int P = 3;
};

__device__ __forceinline__ uint32_t pack2(__nv_bfloat16, float x, float y) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pack2(__half, float x, float y) {
  const __half2 p = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&p);
}

// Two values as the terms' pairs: themselves, or three bfloat16 terms that sum to them.
template <typename T>
__device__ __forceinline__ void terms(float x, float y, uint32_t (&r)[Term<T>::P]) {
  using S = typename Term<T>::type;
  r[0] = pack2(S{}, x, y);
  if constexpr (Term<T>::P == 3) {
#pragma unroll
    for (int p = 1; p < 3; ++p) {
      x -= __uint_as_float(r[p - 1] << 16);  // a bfloat16 is the upper half of a float
      y -= __uint_as_float(r[p - 1] & 0xffff0000u);
      r[p] = pack2(S{}, x, y);
    }
  }
}

// c += a b for the 16 x 8 x 16 product of a warp.
__device__ __forceinline__ void mma(__nv_bfloat16, float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma(__half, float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
               : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
               : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8(uint32_t x) {
  uint32_t y;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}

// The terms' products that count, (term of a, term of b), the smallest first: (2, 0), (0, 2), (1, 1),
// (1, 0), (0, 1), (0, 0), a digit each.
template <int P>
struct Pairs {
  static constexpr int N = P == 3 ? 6 : 1;
  __device__ static constexpr int a(int q) { return P == 3 ? (0x001102 >> (4 * q)) & 3 : 0; }
  __device__ static constexpr int b(int q) { return P == 3 ? (0x010120 >> (4 * q)) & 3 : 0; }
};

// NV neighbouring entries from p on, `n` of them (the others zero); `wide`: p is aligned to a chunk.
template <typename T, int NV>
__device__ __forceinline__ void load_chunk(const T* p, int n, bool wide, float (&x)[NV]) {
  if (wide && n >= NV) {
    if constexpr (sizeof(T) == 4) {
#pragma unroll
      for (int i = 0; i < NV / 4; ++i) {
        const float4 v = __ldcs(reinterpret_cast<const float4*>(p) + i);
        x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
      }
    } else if constexpr (NV == 4) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(p));
      const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
      for (int i = 0; i < 4; ++i) x[i] = to_f32(t[i]);
    } else {
#pragma unroll
      for (int i = 0; i < NV / 8; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(p) + i);
        const T* t = reinterpret_cast<const T*>(&v);
#pragma unroll
        for (int q = 0; q < 8; ++q) x[8 * i + q] = to_f32(t[q]);
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NV; ++i) x[i] = i < n ? to_f32(p[i]) : 0.f;
  }
}
template <typename T, int NV>
__device__ __forceinline__ bool chunk_wide(const T* p, int64_t ld) {
  constexpr int B = NV * sizeof(T) < 16 ? NV * sizeof(T) : 16;
  return ((uintptr_t)p & (B - 1)) == 0 && ld * (int64_t)sizeof(T) % B == 0;
}

// 4 KS neighbouring entries of rows g and g + 8 of a warp's 16: float32 as such, 16-bit types as the
// pairs that the products take.
template <typename T, int KS>
struct Chunk {
  static constexpr int W = sizeof(T) == 4 ? 4 * KS : 2 * KS;
  using type = typename std::conditional<sizeof(T) == 4, float, uint32_t>::type;
  type v[2][W];
  // the entries as float32
  __device__ __forceinline__ void values(float (&x)[2][4 * KS]) const {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int i = 0; i < 4 * KS; ++i) {
        if constexpr (sizeof(T) == 4) x[h][i] = v[h][i];
        else x[h][i] = to_f32(reinterpret_cast<const T*>(&v[h][i / 2])[i % 2]);
      }
  }
};

template <typename T, int KS>
struct Rows {
  const T* p;
  int64_t ld;
  int n;  // entries of the lane's chunk inside the matrix
  bool wide;
  __device__ __forceinline__ Rows(const void* base, int64_t pitch, int cols) : ld(pitch) {
    const int t = threadIdx.x & 3;
    p = static_cast<const T*>(base) + 4 * KS * t;
    n = cols - 4 * KS * t;
    wide = n >= 4 * KS && chunk_wide<T, 4 * KS>(static_cast<const T*>(base), pitch);
  }
  __device__ __forceinline__ void load(int64_t r0, int64_t m, float (&x)[2][4 * KS]) const {
    const int64_t r = r0 + ((threadIdx.x & 31) >> 2);
    load_chunk<T, 4 * KS>(p + r * ld, r < m ? n : 0, wide, x[0]);
    load_chunk<T, 4 * KS>(p + (r + 8) * ld, r + 8 < m ? n : 0, wide, x[1]);
  }
  __device__ __forceinline__ void load(int64_t r0, int64_t m, Chunk<T, KS>& c) const {
    if constexpr (sizeof(T) == 4) {
      load(r0, m, c.v);
    } else {
      const int64_t r1 = r0 + ((threadIdx.x & 31) >> 2);
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int64_t r = r1 + 8 * h;
        const T* q = p + r * ld;
        const int k = r < m ? n : 0;
        if (wide && k > 0) {
          if constexpr (KS == 1) {
            const uint2 v = __ldcs(reinterpret_cast<const uint2*>(q));
            c.v[h][0] = v.x; c.v[h][1] = v.y;
          } else {
#pragma unroll
            for (int i = 0; i < KS / 2; ++i) {
              const uint4 v = __ldcs(reinterpret_cast<const uint4*>(q) + i);
              c.v[h][4 * i] = v.x; c.v[h][4 * i + 1] = v.y; c.v[h][4 * i + 2] = v.z; c.v[h][4 * i + 3] = v.w;
            }
          }
        } else {
          const uint16_t* u = reinterpret_cast<const uint16_t*>(q);
#pragma unroll
          for (int i = 0; i < 2 * KS; ++i)
            c.v[h][i] = (2 * i < k ? (uint32_t)u[2 * i] : 0u) | (2 * i + 1 < k ? (uint32_t)u[2 * i + 1] << 16 : 0u);
        }
      }
    }
  }
};

// The fragments of 16 rows x 16 entries, step s of a chunk: [term][register].
template <typename T, int KS>
__device__ __forceinline__ void fragments(const float (&x)[2][4 * KS], int s, uint32_t (&a)[Term<T>::P][4]) {
#pragma unroll
  for (int h = 0; h < 2; ++h)
#pragma unroll
    for (int p = 0; p < 2; ++p) {
      uint32_t r[Term<T>::P];
      terms<T>(x[h][4 * s + 2 * p], x[h][4 * s + 2 * p + 1], r);
#pragma unroll
      for (int q = 0; q < Term<T>::P; ++q) a[q][h + 2 * p] = r[q];
    }
}
template <typename T, int KS>
__device__ __forceinline__ void fragments(const Chunk<T, KS>& x, int s, uint32_t (&a)[Term<T>::P][4]) {
  if constexpr (sizeof(T) == 4) {
    fragments<T, KS>(x.v, s, a);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll
      for (int p = 0; p < 2; ++p) a[0][h + 2 * p] = x.v[h][2 * s + p];
  }
}

// A matrix (16 KS rows of kk, 8 NT columns, entry (i, j) at p[i * s0 + j * s1], zero beyond rows x cols) as the
// products' second operand: [step][tile][term][lane].
template <typename T, int KS, int NT>
__device__ __forceinline__ void stage_operand(uint2* ws, const T* p, int64_t s0, int64_t s1, int rows, int cols) {
  constexpr int P = Term<T>::P;
#pragma unroll 4
  for (int e = threadIdx.x; e < KS * NT * 32; e += THREADS) {
    const int lane = e & 31, nt = (e >> 5) % NT, s = (e >> 5) / NT, g = lane >> 2, t = lane & 3;
    const int j = 2 * NT * (g >> 1) + 2 * nt + (g & 1), i0 = 4 * KS * t + 4 * s;
    float x[4];
#pragma unroll
    for (int q = 0; q < 4; ++q) x[q] = i0 + q < rows && j < cols ? to_f32(p[(i0 + q) * s0 + j * s1]) : 0.f;
    uint32_t lo[P], hi[P];
    terms<T>(x[0], x[1], lo);
    terms<T>(x[2], x[3], hi);
#pragma unroll
    for (int q = 0; q < P; ++q) ws[((s * NT + nt) * P + q) * 32 + lane] = make_uint2(lo[q], hi[q]);
  }
}

// 16 rows times the staged operand: 2 NT neighbouring results of rows g and g + 8 a lane.
template <typename T, int KS, int NT, typename X>
__device__ __forceinline__ void rows_times(const X& x, const uint2* ws, float (&out)[2][2 * NT]) {
  using S = typename Term<T>::type;
  using PR = Pairs<Term<T>::P>;
  constexpr int P = Term<T>::P;
  const int lane = threadIdx.x & 31;
  float acc[NT][4] = {};
#pragma unroll
  for (int s = 0; s < KS; ++s) {
    uint32_t a[P][4];
    fragments<T, KS>(x, s, a);
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      uint2 b[P];
#pragma unroll
      for (int q = 0; q < P; ++q) b[q] = ws[((s * NT + nt) * P + q) * 32 + lane];
#pragma unroll
      for (int q = 0; q < PR::N; ++q) mma(S{}, acc[nt], a[PR::a(q)], b[PR::b(q)].x, b[PR::b(q)].y);
    }
  }
#pragma unroll
  for (int nt = 0; nt < NT; ++nt) {
    out[0][2 * nt] = acc[nt][0];
    out[0][2 * nt + 1] = acc[nt][1];
    out[1][2 * nt] = acc[nt][2];
    out[1][2 * nt + 1] = acc[nt][3];
  }
}

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

// KN, KC: steps of 16 of the features and of the outputs. DX, DW: which products; dW's comes with db.
// Registers for 4 CTAs a SM (128 a thread) where they suffice, 3 for float32 of 32 x 32 (1,000,000 rows: 99 us; 131 us
// with 4 and its spills), else what it takes.
template <typename T, int KN, int KC>
constexpr int thin_ctas() {
  return KN * KC <= (sizeof(T) == 4 ? 2 : 4) ? 4 : KN * KC <= 4 ? 3 : 1;
}

template <typename T, int KN, int KC, bool DX, bool DW>
__global__ void __launch_bounds__(THREADS, (thin_ctas<T, KN, KC>())) thin_grad_kernel(const ThinArgs a) {
  using S = typename Term<T>::type;
  using PR = Pairs<Term<T>::P>;
  constexpr int P = Term<T>::P;
  __shared__ uint2 ws[DX ? KC * (2 * KN) * P * 32 : 1];
  __shared__ float sums[DW ? WARPS / 2 * (KN * KC * 256 + 32 * 4 * KC) : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  after_previous();
  if constexpr (DX) stage_operand<T, KC, 2 * KN>(ws, static_cast<const T*>(a.W), a.ws1, a.ws0, a.k, a.n);
  __syncthreads();
  const int64_t tiles = (a.m + 15) / 16, step = (int64_t)gridDim.x * WARPS;
  const Rows<T, KC> gr(a.G, a.ldg, a.k), zr(a.Z, a.ldz, a.k);
  const Rows<T, KN> xr(a.X, a.ldx, a.n);
  constexpr int WIDE_DX = 4 * KN < 16 ? 4 * KN : 16;
  T* dx = static_cast<T*>(a.DX) + 4 * KN * t;
  const bool wide_dx = ((uintptr_t)a.DX & 15u) == 0 && a.lddx * (int64_t)sizeof(T) % 16 == 0;
  const int left = a.n - 4 * KN * t;
  float acc[DW ? KN : 1][DW ? 2 * KC : 1][4] = {}, db[DW ? 4 * KC : 1] = {};

  // The next rows are on their way while these are worked on, where the registers allow it (1,000,000 rows:
  // 8 x 8 bfloat16 50 us, 75 without; 32 x 32 100 us, 88 without; float32 32 x 32 197 us, 99 without).
  constexpr bool AHEAD = KN * KC == 1 || (sizeof(T) == 2 && !DW);
  int64_t w = (int64_t)blockIdx.x * WARPS + warp;
  Chunk<T, KC> gn, zn;
  Chunk<T, KN> xn;
  auto fetch = [&](int64_t r0) {
    gr.load(r0, a.m, gn);
    if (DW && a.DW) xr.load(r0, a.m, xn);
    if (a.act != FXTX_ACT_NONE) zr.load(r0, a.m, zn);
  };
  if constexpr (AHEAD) fetch(w * 16);
  for (; w < tiles; w += step) {
    const int64_t r = w * 16 + g;
    float d[2][4 * KC], z[2][4 * KC];
    Chunk<T, KN> x;
    if constexpr (AHEAD) {
      gn.values(d);
      if (a.act != FXTX_ACT_NONE) zn.values(z);
      x = xn;
      fetch((w + step) * 16);
    } else {
      gr.load(w * 16, a.m, d);
      if (DW && a.DW) xr.load(w * 16, a.m, x);
    }
    with_act(a.act, [&](auto act) {
      constexpr int ACT = decltype(act)::value;
      if constexpr (ACT != FXTX_ACT_NONE) {
        if constexpr (!AHEAD) zr.load(w * 16, a.m, z);
#pragma unroll
        for (int h = 0; h < 2; ++h)
#pragma unroll
          for (int i = 0; i < 4 * KC; ++i) d[h][i] *= slope_of<ACT, T>(z[h][i]);
      }
    });
    if constexpr (DX) {
      float c[2][4 * KN];
      rows_times<T, KC, 2 * KN>(d, ws, c);
#pragma unroll
      for (int h = 0; h < 2; ++h)
        if (r + 8 * h < a.m && left > 0) {
#pragma unroll
          for (int i = 0; i < 4 * KN; i += WIDE_DX)
            if (left > i)
              Finish<T>::template store<WIDE_DX>(dx + (r + 8 * h) * a.lddx + i, left - i < WIDE_DX ? left - i : WIDE_DX,
                                                 wide_dx, c[h] + i);
        }
    }
    if constexpr (DW) {
#pragma unroll
      for (int i = 0; i < 4 * KC; ++i) db[i] += d[0][i] + d[1][i];
      if (a.DW) {
        // D's blocks transposed: [step][8 outputs of it][term], rows 0..7 and 8..15
        uint2 dt[KC][2][P];
#pragma unroll
        for (int s = 0; s < KC; ++s) {
          uint32_t f[P][4];
          fragments<T, KC>(d, s, f);
#pragma unroll
          for (int p = 0; p < 2; ++p)
#pragma unroll
            for (int q = 0; q < P; ++q) dt[s][p][q] = make_uint2(transpose8(f[q][2 * p]), transpose8(f[q][2 * p + 1]));
        }
#pragma unroll
        for (int s = 0; s < KN; ++s) {
          uint32_t f[P][4], xt[P][4];
          fragments<T, KN>(x, s, f);
#pragma unroll
          for (int q = 0; q < P; ++q) {
            xt[q][0] = transpose8(f[q][0]);
            xt[q][1] = transpose8(f[q][2]);
            xt[q][2] = transpose8(f[q][1]);
            xt[q][3] = transpose8(f[q][3]);
          }
#pragma unroll
          for (int c = 0; c < 2 * KC; ++c) {
            if constexpr (P == 1) {
              mma(S{}, acc[s][c], xt[0], dt[c / 2][c % 2][0].x, dt[c / 2][c % 2][0].y);
            } else {
              float v[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
              for (int q = 0; q < PR::N; ++q) mma(S{}, v, xt[PR::a(q)], dt[c / 2][c % 2][PR::b(q)].x, dt[c / 2][c % 2][PR::b(q)].y);
#pragma unroll
              for (int i = 0; i < 4; ++i) acc[s][c][i] += v[i];
            }
          }
        }
      }
    }
  }

  if constexpr (DW) {
    // the warps' sums to this CTA's place: the upper half of the warps added to the lower, in turn, as
    // the lanes hold them ([register][lane])
    constexpr int SIZE = KN * KC * 256 + 32 * 4 * KC;
    float* part = a.part + (int64_t)blockIdx.x * SIZE;
#pragma unroll
    for (int half = WARPS / 2; half >= 0; half /= 2) {
      if (half > 0 && warp >= half && warp < 2 * half) {
        float* at = sums + (warp - half) * SIZE + lane;
#pragma unroll
        for (int e = 0; e < KN * KC * 8; ++e) at[e * 32] = acc[e / (8 * KC)][e / 4 % (2 * KC)][e % 4];
#pragma unroll
        for (int i = 0; i < 4 * KC; ++i) at[(KN * KC * 8 + i) * 32] = db[i];
      }
      __syncthreads();
      if (half > 0 ? warp < half : warp == 0) {
        const float* at = sums + warp * SIZE + lane;
#pragma unroll
        for (int e = 0; e < KN * KC * 8; ++e) {
          float& v = acc[e / (8 * KC)][e / 4 % (2 * KC)][e % 4];
          if (half > 0) v += at[e * 32];
          else part[e * 32 + lane] = v;
        }
#pragma unroll
        for (int i = 0; i < 4 * KC; ++i) {
          if (half > 0) db[i] += at[(KN * KC * 8 + i) * 32];
          else part[(KN * KC * 8 + i) * 32 + lane] = db[i];
        }
      }
      if (half == 0) break;
      __syncthreads();
    }
  }
}

// dW and db from the CTAs' sums: a CTA takes 32 registers' worth of one ([register][lane]), 8 threads a place.
template <typename T, int KN, int KC>
__global__ void __launch_bounds__(256) thin_join_kernel(const ThinArgs a, int parts) {
  constexpr int SIZE = KN * KC * 256 + 32 * 4 * KC;
  const int lane = threadIdx.x & 31, y = threadIdx.x >> 5, reg = blockIdx.x;
  __shared__ float sum[8][32];
  float s = 0.f;
  after_previous();
#pragma unroll 8
  for (int p = y; p < parts; p += 8) s += a.part[(int64_t)p * SIZE + reg * 32 + lane];
  sum[y][lane] = s;
  __syncthreads();
  if (y != 0) return;
  for (int q = 1; q < 8; ++q) s += sum[q][lane];
  const int g = lane >> 2, t = lane & 3;
  if (reg < KN * KC * 8) {
    // row g (i < 2) or g + 8 of block (st, c): entry 2 (i / 2) + g % 2 of lane g / 2's chunk, step st
    const int st = reg / (8 * KC), c = reg / 4 % (2 * KC), i = reg % 4;
    const int j = 4 * KN * (g >> 1) + 4 * st + 2 * (i >> 1) + (g & 1);
    const int o = 4 * KC * t + 4 * (c >> 1) + 2 * (c & 1) + (i & 1);
    if (a.DW && j < a.n && o < a.k) static_cast<T*>(a.DW)[j * a.dws0 + o * a.dws1] = from_f32<T>(s);
  } else {
    s += __shfl_xor_sync(FULL_MASK, s, 4);
    s += __shfl_xor_sync(FULL_MASK, s, 8);
    s += __shfl_xor_sync(FULL_MASK, s, 16);
    const int o = 4 * KC * t + reg - KN * KC * 8;
    if (a.DB && g == 0 && o < a.k) static_cast<T*>(a.DB)[o] = from_f32<T>(s);
  }
}

// CTAs of a persistent grid: as many as fit the SMs (asked once a kernel), or as there are rows for.
template <auto KERNEL>
unsigned grid_of(int64_t m, int sm_count) {
  static const int per_sm = [] {
    int b = 0;
    if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, KERNEL, THREADS, 0) != cudaSuccess) cudaGetLastError();
    return std::max(b, 1);
  }();
  return (unsigned)std::min<int64_t>((m + 16 * WARPS - 1) / (16 * WARPS), (int64_t)per_sm * sm_count);
}

template <typename T, int KS, int NT>
cudaError_t launch_layer(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return launch_kernel(thin_kernel<T, KS, NT>, dim3(grid_of<thin_kernel<T, KS, NT>>(a.m, sm_count)), THREADS, 0, st, a);
}

template <typename T, int KN, int KC, bool DX, bool DW>
fxtx_status_t launch_grad(ThinArgs a, int sm_count, cudaStream_t st) {
  unsigned ctas = grid_of<thin_grad_kernel<T, KN, KC, DX, DW>>(a.m, sm_count);
  if (DW && sizeof(T) == 2)
    ctas = (unsigned)std::max<int64_t>(ctas, (a.m + 16 * WARPS * MOST - 1) / (16 * WARPS * MOST));
  constexpr int SIZE = KN * KC * 256 + 32 * 4 * KC;
  if (DW) {
    const fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)ctas * SIZE * 4, st);
    if (s != FXTX_OK) return s;
  }
  cudaError_t e = launch_kernel(thin_grad_kernel<T, KN, KC, DX, DW>, dim3(ctas), THREADS, 0, st, a);
  if (DW) {
    if (e == cudaSuccess) {
      e = launch_kernel(thin_join_kernel<T, KN, KC>, dim3(SIZE / 32), 256, 0, st, a, (int)ctas);
    }
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

// Both products in one pass over G and Z, but for 64 x 64: their registers (128 of dW alone)
// leave too few warps, so they take a pass each.
template <typename T, int KN, int KC>
fxtx_status_t grad_nk(const ThinArgs& a, int sm_count, cudaStream_t st) {
  const bool dw = a.DW || a.DB;
  if constexpr (KN * KC <= 8) {
    if (a.DX && dw) return launch_grad<T, KN, KC, true, true>(a, sm_count, st);
  }
  if (a.DX) {
    const fxtx_status_t s = launch_grad<T, KN, KC, true, false>(a, sm_count, st);
    if (s != FXTX_OK) return s;
  }
  return dw ? launch_grad<T, KN, KC, false, true>(a, sm_count, st) : FXTX_OK;
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

template <typename T, int KN>
fxtx_status_t grad_k(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return a.k <= 16 ? grad_nk<T, KN, 1>(a, sm_count, st)
                   : a.k <= 32 ? grad_nk<T, KN, 2>(a, sm_count, st) : grad_nk<T, KN, 4>(a, sm_count, st);
}
template <typename T>
fxtx_status_t grad_t(const ThinArgs& a, int sm_count, cudaStream_t st) {
  return a.n <= 16 ? grad_k<T, 1>(a, sm_count, st)
                   : a.n <= 32 ? grad_k<T, 2>(a, sm_count, st) : grad_k<T, 4>(a, sm_count, st);
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
    case FXTX_F32: return grad_t<float>(a, dev.sm_count, st);
    case FXTX_BF16: return grad_t<__nv_bfloat16>(a, dev.sm_count, st);
    default: return grad_t<__half>(a, dev.sm_count, st);
  }
}

}  // namespace fxtx
