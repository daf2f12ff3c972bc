// norm.cu — layer norm over the rows of X and its gradient:
//     out = u w + b,  u = (x - mean) rstd,  rstd = (mean of (x - mean)^2 + eps)^-1/2
//     h = g w:  dx = rstd (h - mean(h) - u mean(h u)) + r,  dw = sum over the rows of g u,  db = of g
//
// Bound: HBM; every matrix is read or written once. A row lies in the registers of `tpr` threads (1 to 32 neighbouring
// lanes, or whole warps that meet at a named barrier), CH accesses of 16 bytes each, so that the variance is formed
// from x - mean without reading x again. A CTA has `groups` such rows in work at once and takes rows in turn. The columns of a
// thread stay the same from row to row, so dw and db are summed in its registers, over the CTA's groups in shared memory, in
// turn, and over the CTAs by a second kernel in order: the result is the same on every call.
//
// Which kernel, by the rows' number, width and alignment (bytes in all: 16384 x 4096 bfloat16 268 MB forward, 537 MB backward with
// the residual path; 1,000,000 x 32 float32 384 MB backward):
//   norm_ring_kernel, norm_grad_ring_kernel   many rows of more than a warp's accesses: bulk copies bring a group's next rows into a
//              ring; 48 us (5.6 TB/s: the instructions of 16 warps a SM) and 85 us (6.3 TB/s); the register kernels 57 and 138 us
//   norm_grad_short_kernel   many rows of at most 32 accesses: a ring of tiles a warp; 68 us (5.6 TB/s), in registers 90
//   norm_odd_kernel, norm_grad_odd_kernel   many rows whose pitch or width is no multiple of 16 bytes, of 129 to 8,192 entries;
//              30,001 x 2047 bfloat16 108 and 152 us (177 with the residual path), entry by entry from memory 218 and 564
//   norm_kernel, norm_grad_kernel   the others: rows loaded into registers, the next one ahead; one row of 4096 3.3 us
//   norm_long_kernel and norm_long_means_kernel, norm_long_grad_kernel   rows beyond what the registers hold (16 bits: 32,768
//              forward, 8,192 backward; float32 half and the same): x read three times, one CTA a row; backward the two means in
//              one pass, dx and the column sums in another
// Rows that go entry by entry (V = 1) have neighbouring threads take neighbouring entries.
#include <algorithm>
#include <atomic>
#include <type_traits>

#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "ring.h"
#include "train.h"

namespace fxtx {

int* norm_error_word() { return device_error_word(); }

namespace {

constexpr int FWD_THREADS = 256, GRAD_THREADS = 512, LONG_THREADS = 512;

__device__ __forceinline__ uint32_t pair(__nv_bfloat16, float x, float y) {
  const __nv_bfloat162 p = __floats2bfloat162_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ uint32_t pair(__half, float x, float y) {
  const __half2 p = __floats2half2_rn(x, y);
  return *reinterpret_cast<const uint32_t*>(&p);
}
__device__ __forceinline__ float2 unpair(__nv_bfloat16, uint32_t v) { return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u)); }
__device__ __forceinline__ float2 unpair(__half, uint32_t v) { return __half22float2(*reinterpret_cast<const __half2*>(&v)); }

// Two values in one register pair, and their operations, an instruction for both.
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
__device__ __forceinline__ f2 mul2(f2 a, f2 b) {
  f2 r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ __forceinline__ f2 fma2(f2 a, f2 b, f2 c) {
  f2 r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}

// V neighbouring entries as they are loaded.
template <typename T, int V>
struct Raw {
  static_assert(V * sizeof(T) == 16, "16 bytes");
  uint4 v;
  __device__ __forceinline__ void load(const T* p) { v = *reinterpret_cast<const uint4*>(p); }
  __device__ __forceinline__ void zero() { v = make_uint4(0, 0, 0, 0); }
  __device__ __forceinline__ void values(float* x) const {
    const uint32_t t[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if constexpr (V == 4) {
        x[i] = __uint_as_float(t[i]);
      } else {
        const float2 y = unpair(T{}, t[i]);
        x[2 * i] = y.x;
        x[2 * i + 1] = y.y;
      }
    }
  }
  __device__ __forceinline__ void pairs(f2* x) const {
    float y[V];
    values(y);
#pragma unroll
    for (int i = 0; i < V / 2; ++i) x[i] = pack2(y[2 * i], y[2 * i + 1]);
  }
  __device__ __forceinline__ static void store_pairs(T* p, const f2* x) {
    float y[V];
#pragma unroll
    for (int i = 0; i < V / 2; ++i) {
      const float2 v = unpack2(x[i]);
      y[2 * i] = v.x;
      y[2 * i + 1] = v.y;
    }
    store(p, y);
  }
  __device__ __forceinline__ static void store(T* p, const float* x) {
    uint4 w;
    if constexpr (V == 4) {
      w = make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]), __float_as_uint(x[3]));
    } else {  // two at a time, an instruction each
      w = make_uint4(pair(T{}, x[0], x[1]), pair(T{}, x[2], x[3]), pair(T{}, x[4], x[5]), pair(T{}, x[6], x[7]));
    }
    *reinterpret_cast<uint4*>(p) = w;
  }
};
template <typename T>
struct Raw<T, 1> {
  T v;
  __device__ __forceinline__ void load(const T* p) { v = *p; }
  __device__ __forceinline__ void zero() { v = from_f32<T>(0.f); }
  __device__ __forceinline__ void values(float* x) const { x[0] = to_f32(v); }
  __device__ __forceinline__ static void store(T* p, const float* x) { *p = from_f32<T>(x[0]); }
};

// How rows lie over a CTA's threads.
struct RowShape {
  int tpr = 1, groups = 1;
};

// A row's accesses: thread t of its tpr takes accesses t, t + tpr, ...
template <typename T, int V, int CH>
struct RowOf {
  const int t, tpr, count;
  __device__ __forceinline__ RowOf(int t_, int tpr_, int64_t n) : t(t_), tpr(tpr_), count((int)(n / V)) {}
  __device__ __forceinline__ bool has(int i) const { return t + i * tpr < count; }
  __device__ __forceinline__ int64_t at(int i) const { return (int64_t)(t + i * tpr) * V; }
  __device__ __forceinline__ void load(const void* base, int64_t row, int64_t rows, int64_t ld, Raw<T, V> (&x)[CH]) const {
    const T* p = static_cast<const T*>(base) + row * ld;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (row < rows && has(i)) x[i].load(p + at(i));
      else x[i].zero();
    }
  }
};

// A row's whole warps meet.
__device__ __forceinline__ void group_barrier(int group, int tpr) { asm volatile("bar.sync %0, %1;" ::"r"(group + 1), "r"(tpr) : "memory"); }

// Sums over a row's threads, the same in each of them. All threads of the CTA call it as often.
template <bool BIG>
struct RowSum {
  float2 (*red)[32];  // [2][warps of the CTA]
  int tpr, group, parity = 0;
  __device__ __forceinline__ float2 operator()(float2 s) {
    if constexpr (!BIG) {
      for (int o = tpr >> 1; o > 0; o >>= 1) {
        s.x += shfl_xor(s.x, o);
        s.y += shfl_xor(s.y, o);
      }
      return s;
    } else {
      s.x = group_sum<32>(s.x);
      s.y = group_sum<32>(s.y);
      const int warp = threadIdx.x >> 5, w0 = group * (tpr >> 5), wn = tpr >> 5;
      float2* buf = red[parity];
      parity ^= 1;  // whoever writes this half again has passed the other half's barrier, which all readers of this one reach after
      if ((threadIdx.x & 31) == 0) buf[warp] = s;
      group_barrier(group, tpr);
      s = make_float2(0.f, 0.f);
      for (int w = 0; w < wn; ++w) {
        const float2 v = buf[w0 + w];
        s.x += v.x;
        s.y += v.y;
      }
      return s;
    }
  }
};

template <typename T, int V, int CH, bool BIG>
__global__ void __launch_bounds__(1024) norm_kernel(const __grid_constant__ NormArgs a, const RowShape shape) {
  __shared__ float2 red[2][32];
  const int tpr = shape.tpr, group = threadIdx.x / tpr;
  const RowOf<T, V, CH> r((int)threadIdx.x % tpr, tpr, a.n);
  RowSum<BIG> sum{red, tpr, group};
  const float over = 1.f / (float)a.n;
  const int64_t step = (int64_t)gridDim.x * shape.groups;
  int64_t row = (int64_t)blockIdx.x * shape.groups + group;
  after_previous();
  Raw<T, V> next[CH];
  r.load(a.X, row, a.m, a.ldx, next);
  // (all threads go round as often as the CTA's first group, whose rows are the lowest)
  for (int64_t first = (int64_t)blockIdx.x * shape.groups; first < a.m; first += step, row += step) {
    float x[CH * V];
#pragma unroll
    for (int i = 0; i < CH; ++i) next[i].values(x + i * V);
    r.load(a.X, row + step, a.m, a.ldx, next);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CH * V; ++i) s += x[i];
    const float mean = sum(make_float2(s, 0.f)).x * over;
    s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (r.has(i)) {
#pragma unroll
        for (int q = 0; q < V; ++q) {
          float& v = x[i * V + q];
          v -= mean;
          s = fmaf(v, v, s);
        }
      }
    const float rstd = __frsqrt_rn(fmaf(sum(make_float2(s, 0.f)).x, over, a.eps));
    if (row >= a.m) continue;
    if (r.t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* out = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!r.has(i)) continue;
      float* v = x + i * V;
#pragma unroll
      for (int q = 0; q < V; ++q) v[q] *= rstd;
      Raw<T, V> c;
      float y[V];
      if (a.w) {
        c.load(static_cast<const T*>(a.w) + r.at(i));
        c.values(y);
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] *= y[q];
      }
      if (a.b) {
        c.load(static_cast<const T*>(a.b) + r.at(i));
        c.values(y);
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] += y[q];
      }
      Raw<T, V>::store(out + r.at(i), v);
    }
  }
}

// SUMS: dw and db too.
template <typename T, int V, int CH, bool BIG, bool SUMS>
__global__ void __launch_bounds__(GRAD_THREADS, 1) norm_grad_kernel(const __grid_constant__ NormArgs a, const RowShape shape) {
  __shared__ float2 red[2][32];
  constexpr int E = CH * V;
  const int tpr = shape.tpr, group = threadIdx.x / tpr;
  const RowOf<T, V, CH> r((int)threadIdx.x % tpr, tpr, a.n);
  RowSum<BIG> sum{red, tpr, group};
  const float over = 1.f / (float)a.n;
  const int64_t step = (int64_t)gridDim.x * shape.groups;
  int64_t row = (int64_t)blockIdx.x * shape.groups + group;
  after_previous();
  float dw[SUMS ? E : 1] = {}, db[SUMS ? E : 1] = {};
  Raw<T, V> w[CH], xn[CH], gn[CH], rn[CH];
  if (a.w) r.load(a.w, 0, 1, 0, w);
  float mean_n = 0.f, rstd_n = 0.f;
  auto fetch = [&](int64_t i) {
    r.load(a.X, i, a.m, a.ldx, xn);
    r.load(a.G, i, a.m, a.ldg, gn);
    if (a.R) r.load(a.R, i, a.m, a.ldr, rn);
    mean_n = i < a.m ? a.mean_in[i] : 0.f;
    rstd_n = i < a.m ? a.rstd_in[i] : 0.f;
  };
  fetch(row);
  for (int64_t first = (int64_t)blockIdx.x * shape.groups; first < a.m; first += step, row += step) {
    float u[E], h[E];
    Raw<T, V> res[CH];
    const float mean = mean_n, rstd = rstd_n;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      xn[i].values(u + i * V);
      gn[i].values(h + i * V);
      if (a.R) res[i] = rn[i];
    }
    fetch(row + step);
    float2 s = make_float2(0.f, 0.f);
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      float y[V];
      w[i].values(y);
      // (a thread beyond the row's end, or a row beyond the last, has zeros in G, but for u: those would be no
      // numbers where mean or rstd is none)
      const bool in = r.has(i) && row < a.m;
#pragma unroll
      for (int q = 0; q < V; ++q) {
        float &x = u[i * V + q], &g = h[i * V + q];
        x = in ? (x - mean) * rstd : 0.f;
        if constexpr (SUMS) {
          dw[i * V + q] = fmaf(g, x, dw[i * V + q]);
          db[i * V + q] += g;
        }
        if (a.w) g *= y[q];
        s.x += g;
        s.y = fmaf(g, x, s.y);
      }
    }
    s = sum(s);
    if (row >= a.m || !a.DX) continue;
    const float c1 = s.x * over, c2 = s.y * over;
    T* out = static_cast<T*>(a.DX) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!r.has(i)) continue;
      float v[V], y[V];
      if (a.R) res[i].values(y);
#pragma unroll
      for (int q = 0; q < V; ++q) {
        v[q] = (h[i * V + q] - c1 - u[i * V + q] * c2) * rstd;
        if (a.R) v[q] += y[q];
      }
      Raw<T, V>::store(out + r.at(i), v);
    }
  }
  if constexpr (SUMS) {
    // over the CTA's rows in work: a warp's by exchange, then group after group (or warp after warp) in shared memory
    extern __shared__ __align__(16) float cols[];  // [2][E][tpr]
    if constexpr (!BIG) {
      for (int o = tpr; o < 32; o <<= 1) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          dw[e] += shfl_xor(dw[e], o);
          db[e] += shfl_xor(db[e], o);
        }
      }
    }
    const int units = BIG ? shape.groups : (int)(blockDim.x >> 5), unit = BIG ? group : (int)(threadIdx.x >> 5);
    const bool mine = BIG || (int)(threadIdx.x & 31) < tpr;
    for (int y = 0; y < units; ++y) {
      __syncthreads();
      if (unit != y || !mine) continue;
#pragma unroll
      for (int e = 0; e < E; ++e) {
        float *p = cols + e * tpr + r.t, *q = p + E * tpr;
        *p = y > 0 ? *p + dw[e] : dw[e];
        *q = y > 0 ? *q + db[e] : db[e];
      }
    }
    __syncthreads();
    for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
      const int c = (int)(j / V), e = c / tpr * V + (int)(j % V);
      const float x = cols[e * tpr + c % tpr], y = cols[(E + e) * tpr + c % tpr];
      if (gridDim.x == 1) {
        if (a.DW) static_cast<T*>(a.DW)[j] = from_f32<T>(x);
        if (a.DB) static_cast<T*>(a.DB)[j] = from_f32<T>(y);
      } else {
        float* p = a.part + (int64_t)blockIdx.x * 2 * a.n + j;
        p[0] = x;
        p[a.n] = y;
      }
    }
  }
}

// ------------------------------------------------------------------------------------------------ rows by bulk copies
// Many rows of several warps each: a group's next rows come to a ring in shared memory, several on their way at a time (held
// in registers, one: 8192 rows a group in turn left the memory waiting for the sums).

constexpr int RING_THREADS = 512, RING_BYTES = 200 * 1024, MOST_STAGES = 8, MOST_GROUPS = 8;

__device__ __forceinline__ void copy_row(void* dst, const void* src, uint32_t bytes, uint64_t* bar) {
  asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(smem_addr(dst)), "l"(src),
               "r"(bytes), "r"(smem_addr(bar))
               : "memory");
}

// A warp's wait that gave up (FXTX_ERR_TIMEOUT is raised) ends its rows: nothing more is read, copied or stored. The copying thread
// then waits, each time with a limit, for the copies under way, before anything else is done with their memory,
template <typename I>
__device__ __forceinline__ void drain(uint64_t* full, const RingTurn& turn, I item, I items, I step) {
#pragma unroll 1
  for (int x = 0; x < turn.stages; ++x)
    if (turn.asked(x, item, items, step)) mbar_wait_bounded(&full[x], turn.parity(x));
}
// and the warp meets its group's others at the barriers of the rows that are left.
template <int BARRIERS, typename Ring>
__device__ __forceinline__ void leave_rows(const Ring& ring, bool copies, int group, int tpr, int64_t row, int64_t rows, int64_t step) {
  if (copies) drain(ring.full, ring.turn, row, rows, step);
  __syncwarp();
#pragma unroll 1
  for (; row < rows; row += step)
    for (int i = 0; i < BARRIERS; ++i) group_barrier(group, tpr);
}

// A group's ring: MATS rows (of as many matrices) a stage.
template <typename T, int MATS>
struct RowRing {
  unsigned char* at;   // the group's stages
  uint64_t* full;
  uint32_t bytes;      // of a row
  int mats;
  RingTurn turn;
  __device__ __forceinline__ RowRing(unsigned char* smem, uint64_t* bars, int group, int stages_, int mats_, int64_t n)
      : bytes((uint32_t)(n * sizeof(T))), mats(mats_), turn(stages_) {
    at = smem + (size_t)group * stages_ * mats * bytes;
    full = bars + group * MOST_STAGES;
  }
  __device__ __forceinline__ const T* row(int mat) const { return reinterpret_cast<const T*>(at + (size_t)(turn.s * mats + mat) * bytes); }
  // one thread's: the rows at p[0 .. mats - 1] to stage x
  __device__ __forceinline__ void fill(int x, const void* const (&p)[MATS]) {
    mbar_arrive_expect_tx(&full[x], bytes * (uint32_t)mats);
#pragma unroll
    for (int i = 0; i < MATS; ++i)
      if (i < mats) copy_row(at + (size_t)(x * mats + i) * bytes, p[i], bytes, &full[x]);
  }
  // this turn's copies; false (the whole warp's) after a timeout
  __device__ __forceinline__ bool wait() { return __all_sync(FULL_MASK, mbar_wait_bounded(&full[turn.s], turn.phase)); }
};

// A thread's accesses of a row in shared memory, and of w or b (`none` where there is no such vector).
template <typename T, int V, int CH>
__device__ __forceinline__ void load_pairs(const RowOf<T, V, CH>& r, const T* row, f2* x) {
  Raw<T, V> raw[CH];
  r.load(row, 0, 1, 0, raw);
#pragma unroll
  for (int i = 0; i < CH; ++i) raw[i].pairs(x + i * V / 2);
}
template <typename T, int V, int CH>
__device__ __forceinline__ void load_vector(const RowOf<T, V, CH>& r, const void* p, float none, f2* x) {
  if (p) {
    load_pairs<T, V, CH>(r, static_cast<const T*>(p), x);
  } else {
#pragma unroll
    for (int i = 0; i < CH * V / 2; ++i) x[i] = pack2(none, none);
  }
}

template <typename T, int CH>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_ring_kernel(const __grid_constant__ NormArgs a, const RowShape shape, int stages) {
  constexpr int V = 16 / sizeof(T);
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[MOST_GROUPS * MOST_STAGES];
  __shared__ float2 red[2][32];
  __shared__ float s_n[32];
  const int tpr = shape.tpr, group = threadIdx.x / tpr;
  const RowOf<T, V, CH> r((int)threadIdx.x % tpr, tpr, a.n);
  RowRing<T, 1> ring(smem, full, group, stages, 1, a.n);
  // entries of the thread, of warp y of the row, and of the thread's warp
  const int accesses = (int)(a.n / V);
  auto n_of = [&](int y) {  // whole accesses of 32 threads, and a last one of fewer
    int n = 0;
#pragma unroll
    for (int i = 0; i < CH; ++i) n += min(32, max(0, accesses - y * 32 - i * tpr));
    return (float)(n * V);
  };
  float n_own = 0.f;
#pragma unroll
  for (int i = 0; i < CH; ++i) n_own += r.has(i) ? (float)V : 0.f;
  const float over_own = n_own > 0.f ? 1.f / n_own : 0.f, n_warp = n_of(r.t >> 5), over_warp = n_warp > 0.f ? 1.f / n_warp : 0.f;
  if ((threadIdx.x & 31) == 0) s_n[threadIdx.x >> 5] = n_warp;
  int parity = 0;
  if (r.t == 0) {
    for (int x = 0; x < stages; ++x) mbar_init(&ring.full[x], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const float over = 1.f / (float)a.n;
  const int64_t step = (int64_t)gridDim.x * shape.groups;
  int64_t row = (int64_t)blockIdx.x * shape.groups + group;
  after_previous();
  auto fill = [&](int x, int64_t i) {
    const void* p[1] = {static_cast<const T*>(a.X) + i * a.ldx};
    if (i < a.m) ring.fill(x, p);
  };
  if (r.t == 0)
    for (int x = 0; x < stages; ++x) fill(x, row + x * step);
  constexpr int P = CH * V / 2;  // pairs
  f2 w[P], b[P];
  load_vector<T, V, CH>(r, a.w, 1.f, w);
  load_vector<T, V, CH>(r, a.b, 0.f, b);
  for (; row < a.m; row += step) {
    if (!ring.wait()) break;
    f2 x[P];
    load_pairs<T, V, CH>(r, ring.row(0), x);
    // the thread's own mean and squares about it, the warp's from those, the row's from the warps' (one barrier a row)
    f2 sum = 0, squares = 0;
#pragma unroll
    for (int i = 0; i < P; ++i) sum = add2(sum, x[i]);
    const float own = (unpack2(sum).x + unpack2(sum).y) * over_own;
    const f2 off = pack2(-own, -own);
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (r.has(i)) {
#pragma unroll
        for (int q = 0; q < V / 2; ++q) {
          const f2 v = add2(x[i * V / 2 + q], off);
          squares = fma2(v, v, squares);
        }
      }
    const float warp_mean = group_sum<32>(own * n_own) * over_warp, d = own - warp_mean;
    const float warp_square = group_sum<32>(fmaf(n_own * d, d, unpack2(squares).x + unpack2(squares).y));
    float2* buf = red[parity];
    parity ^= 1;
    if ((threadIdx.x & 31) == 0) buf[threadIdx.x >> 5] = make_float2(warp_mean, warp_square);
    group_barrier(group, tpr);
    // (every thread of the group has read the row)
    if (r.t == 0) fill(ring.turn.s, row + stages * step);
    ring.turn.next();
    const int w0 = group * (tpr >> 5), wn = tpr >> 5;
    float mean = 0.f, square = 0.f;
    for (int y = 0; y < wn; ++y) mean = fmaf(buf[w0 + y].x, s_n[w0 + y], mean);
    mean *= over;
    for (int y = 0; y < wn; ++y) {
      const float2 z = buf[w0 + y];
      square += fmaf(s_n[w0 + y] * (z.x - mean), z.x - mean, z.y);
    }
    const float rstd = __frsqrt_rn(fmaf(square, over, a.eps));
    if (r.t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* out = static_cast<T*>(a.out) + row * a.ldo;
    const f2 minus = pack2(-mean, -mean), scale = pack2(rstd, rstd);
#pragma unroll
    for (int i = 0; i < P; ++i) x[i] = fma2(mul2(add2(x[i], minus), scale), w[i], b[i]);
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (r.has(i)) Raw<T, V>::store_pairs(out + r.at(i), x + i * V / 2);
  }
  leave_rows<1>(ring, r.t == 0, group, tpr, row, a.m, step);
}

// A thread's column sums, over the groups in turn, to the CTA's part (or dw and db, of one CTA).
template <typename T, int V, int CH>
__device__ __forceinline__ void store_columns(const NormArgs& a, const RowOf<T, V, CH>& r, int group, int groups, const float* dw,
                                              const float* db, float* cols) {
  constexpr int E = CH * V;
  for (int y = 0; y < groups; ++y) {
    __syncthreads();
    if (group != y) continue;
#pragma unroll
    for (int e = 0; e < E; ++e) {
      float *p = cols + e * r.tpr + r.t, *q = p + E * r.tpr;
      *p = y > 0 ? *p + dw[e] : dw[e];
      *q = y > 0 ? *q + db[e] : db[e];
    }
  }
  __syncthreads();
  for (int64_t j = threadIdx.x; j < a.n; j += blockDim.x) {
    const int c = (int)(j / V), e = c / r.tpr * V + (int)(j % V);
    const float x = cols[e * r.tpr + c % r.tpr], y = cols[(E + e) * r.tpr + c % r.tpr];
    if (gridDim.x == 1) {
      if (a.DW) static_cast<T*>(a.DW)[j] = from_f32<T>(x);
      if (a.DB) static_cast<T*>(a.DB)[j] = from_f32<T>(y);
    } else {
      float* p = a.part + (int64_t)blockIdx.x * 2 * a.n + j;
      p[0] = x;
      p[a.n] = y;
    }
  }
}

template <typename T, int CH, bool SUMS>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_grad_ring_kernel(const __grid_constant__ NormArgs a, const RowShape shape, int stages) {
  constexpr int V = 16 / sizeof(T), E = CH * V;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[MOST_GROUPS * MOST_STAGES];
  __shared__ float2 red[2][32];
  const int tpr = shape.tpr, group = threadIdx.x / tpr;
  const RowOf<T, V, CH> r((int)threadIdx.x % tpr, tpr, a.n);
  RowSum<true> sum{red, tpr, group};
  RowRing<T, 3> ring(smem, full, group, stages, a.R ? 3 : 2, a.n);
  if (r.t == 0) {
    for (int x = 0; x < stages; ++x) mbar_init(&ring.full[x], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const float over = 1.f / (float)a.n;
  const int64_t step = (int64_t)gridDim.x * shape.groups;
  int64_t row = (int64_t)blockIdx.x * shape.groups + group;
  after_previous();
  auto fill = [&](int x, int64_t i) {
    const void* p[3] = {static_cast<const T*>(a.X) + i * a.ldx, static_cast<const T*>(a.G) + i * a.ldg, static_cast<const T*>(a.R) + i * a.ldr};
    if (i < a.m) ring.fill(x, p);
  };
  if (r.t == 0)
    for (int x = 0; x < stages; ++x) fill(x, row + x * step);
  constexpr int P = E / 2;  // pairs
  f2 dw[SUMS ? P : 1] = {}, db[SUMS ? P : 1] = {}, w[P];
  load_vector<T, V, CH>(r, a.w, 1.f, w);
  float mean_n = row < a.m ? a.mean_in[row] : 0.f, rstd_n = row < a.m ? a.rstd_in[row] : 0.f;
  for (; row < a.m; row += step) {
    const float mean = mean_n, rstd = rstd_n;
    if (row + step < a.m) {
      mean_n = a.mean_in[row + step];
      rstd_n = a.rstd_in[row + step];
    }
    if (!ring.wait()) break;
    f2 u[P], h[P];
    Raw<T, V> res[CH];
    load_pairs<T, V, CH>(r, ring.row(0), u);
    load_pairs<T, V, CH>(r, ring.row(1), h);
    if (a.R) r.load(ring.row(2), 0, 1, 0, res);
    const f2 minus = pack2(-mean, -mean), scale = pack2(rstd, rstd);
    f2 s1 = 0, s2 = 0;
    // (beyond the row's end x and g are zero, and mean is taken as zero there: -mean rstd may be beyond fp32 where u is not)
#pragma unroll
    for (int i = 0; i < P; ++i) {
      u[i] = mul2(add2(u[i], r.has(i / (V / 2)) ? minus : 0), scale);
      if constexpr (SUMS) {
        dw[i] = fma2(h[i], u[i], dw[i]);
        db[i] = add2(db[i], h[i]);
      }
      h[i] = mul2(h[i], w[i]);
      s1 = add2(s1, h[i]);
      s2 = fma2(h[i], u[i], s2);
    }
    const float2 s = sum(make_float2(unpack2(s1).x + unpack2(s1).y, unpack2(s2).x + unpack2(s2).y));
    if (r.t == 0) fill(ring.turn.s, row + stages * step);
    ring.turn.next();
    if (!a.DX) continue;
    const float c1 = -s.x * over, c2 = -s.y * over;
    const f2 d1 = pack2(c1, c1), d2 = pack2(c2, c2);
    T* out = static_cast<T*>(a.DX) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      if (!r.has(i)) continue;
      f2 v[V / 2], y[V / 2];
      if (a.R) {
        res[i].pairs(y);
      } else {
#pragma unroll
        for (int q = 0; q < V / 2; ++q) y[q] = 0;
      }
#pragma unroll
      for (int q = 0; q < V / 2; ++q) v[q] = fma2(fma2(u[i * V / 2 + q], d2, add2(h[i * V / 2 + q], d1)), scale, y[q]);
      Raw<T, V>::store_pairs(out + r.at(i), v);
    }
  }
  leave_rows<1>(ring, r.t == 0, group, tpr, row, a.m, step);
  if constexpr (SUMS) {
    float x[E], y[E];
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[2 * i] = unpack2(dw[i]).x;
      x[2 * i + 1] = unpack2(dw[i]).y;
      y[2 * i] = unpack2(db[i]).x;
      y[2 * i + 1] = unpack2(db[i]).y;
    }
    store_columns<T, V, CH>(a, r, group, shape.groups, x, y, reinterpret_cast<float*>(smem));
  }
}

// ------------------------------------------------------------------------------------------------ rows of any width by bulk copies
// Many rows whose pitch or width is no multiple of 16 bytes, from 16-byte aligned matrices: a row comes with what of its first
// and last 16 bytes belongs to its neighbours (of the last row the end is read where it lies), and threads take its entries
// from shared memory, neighbours neighbouring ones (entry by entry from memory, 30,001 x 2047 bfloat16 took 218 us, its
// gradient 564).

template <typename T, int MATS>
struct OddRing {
  unsigned char* at;
  uint64_t* full;
  int slot, mats;
  RingTurn turn;
  __device__ __forceinline__ OddRing(unsigned char* smem, uint64_t* bars, int group, int slot_, int stages_, int mats_)
      : slot(slot_), mats(mats_), turn(stages_) {
    at = smem + (size_t)group * stages_ * mats * slot;
    full = bars + group * MOST_STAGES;
  }
  // where a row's copy begins, and its bytes
  __device__ __forceinline__ static uint32_t head(const T* p) { return (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u); }
  __device__ __forceinline__ static uint32_t copied(const T* p, int64_t n, bool last) {
    const uint32_t bytes = head(p) + (uint32_t)(n * sizeof(T));
    return last ? bytes / 16 * 16 : (bytes + 15) / 16 * 16;
  }
  __device__ __forceinline__ void fill(int x, const T* const (&p)[MATS], int64_t n, bool last) {
    uint32_t all = 0;
#pragma unroll
    for (int i = 0; i < MATS; ++i)
      if (i < mats) all += copied(p[i], n, last);
    mbar_arrive_expect_tx(&full[x], all);
#pragma unroll
    for (int i = 0; i < MATS; ++i)
      if (i < mats) {
        const uint32_t bytes = copied(p[i], n, last);
        if (bytes) copy_row(at + (size_t)(x * mats + i) * slot, reinterpret_cast<const unsigned char*>(p[i]) - head(p[i]), bytes, &full[x]);
      }
  }
  // this turn's copies; false (the whole warp's) after a timeout
  __device__ __forceinline__ bool wait() { return __all_sync(FULL_MASK, mbar_wait_bounded(&full[turn.s], turn.phase)); }
  // the thread's entries of the row at p
  // (`beyond` for what lies beyond its end)
  template <int CH>
  __device__ __forceinline__ void load(int mat, const T* p, int t, int tpr, int n, bool last, float (&x)[CH], float beyond = 0.f) const {
    const T* row = reinterpret_cast<const T*>(at + (size_t)(turn.s * mats + mat) * slot + head(p));
    if (!last) {
#pragma unroll
      for (int i = 0; i < CH; ++i) {
        const int j = t + i * tpr;
        x[i] = to_f32(row[j < n ? j : 0]);
        if (j >= n) x[i] = beyond;
      }
      return;
    }
    const int there = (int)((max(copied(p, n, true), head(p)) - head(p)) / sizeof(T));
#pragma unroll 1
    for (int i = 0; i < CH; ++i) {
      const int j = t + i * tpr;
      const float v = j < there ? to_f32(row[j]) : j < n ? to_f32(p[j]) : beyond;
#pragma unroll
      for (int q = 0; q < CH; ++q) x[q] = q == i ? v : x[q];
    }
  }
};

template <typename T, int CH>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_odd_kernel(const __grid_constant__ NormArgs a, const RowShape shape, int slot, int stages) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[MOST_GROUPS * MOST_STAGES];
  __shared__ float2 red[2][32];
  const int tpr = shape.tpr, group = threadIdx.x / tpr, t = threadIdx.x % tpr, n = (int)a.n;
  RowSum<true> sum{red, tpr, group};
  OddRing<T, 1> ring(smem, full, group, slot, stages, 1);
  if (t == 0) {
    for (int x = 0; x < stages; ++x) mbar_init(&ring.full[x], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const float over = 1.f / (float)n;
  const int64_t step = (int64_t)gridDim.x * shape.groups;
  int64_t row = (int64_t)blockIdx.x * shape.groups + group;
  after_previous();
  auto at = [&](int64_t i) { return static_cast<const T*>(a.X) + i * a.ldx; };
  auto fill = [&](int x, int64_t i) {
    const T* p[1] = {at(i)};
    if (i < a.m) ring.fill(x, p, n, i + 1 == a.m);
  };
  if (t == 0)
    for (int x = 0; x < stages; ++x) fill(x, row + x * step);
  float w[CH], b[CH];
#pragma unroll
  for (int i = 0; i < CH; ++i) {
    const int j = t + i * tpr;
    w[i] = a.w && j < n ? to_f32(static_cast<const T*>(a.w)[j]) : 1.f;
    b[i] = a.b && j < n ? to_f32(static_cast<const T*>(a.b)[j]) : 0.f;
  }
  for (; row < a.m; row += step) {
    if (!ring.wait()) break;
    float x[CH];
    ring.load(0, at(row), t, tpr, n, row + 1 == a.m, x);
    float s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) s += x[i];
    const float mean = sum(make_float2(s, 0.f)).x * over;
    // (every thread of the group has read the row)
    if (t == 0) fill(ring.turn.s, row + stages * step);
    ring.turn.next();
    s = 0.f;
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      x[i] = t + i * tpr < n ? x[i] - mean : 0.f;
      s = fmaf(x[i], x[i], s);
    }
    const float rstd = __frsqrt_rn(fmaf(sum(make_float2(s, 0.f)).x, over, a.eps));
    if (t == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* out = static_cast<T*>(a.out) + row * a.ldo;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (t + i * tpr < n) out[t + i * tpr] = from_f32<T>(fmaf(x[i] * rstd, w[i], b[i]));
  }
  leave_rows<2>(ring, t == 0, group, tpr, row, a.m, step);
}

template <typename T, int CH, bool SUMS>
__global__ void __launch_bounds__(RING_THREADS, 1) norm_grad_odd_kernel(const __grid_constant__ NormArgs a, const RowShape shape, int slot,
                                                                       int stages) {
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t full[MOST_GROUPS * MOST_STAGES];
  __shared__ float2 red[2][32];
  const int tpr = shape.tpr, group = threadIdx.x / tpr, t = threadIdx.x % tpr, n = (int)a.n;
  RowSum<true> sum{red, tpr, group};
  OddRing<T, 3> ring(smem, full, group, slot, stages, a.R ? 3 : 2);
  if (t == 0) {
    for (int x = 0; x < stages; ++x) mbar_init(&ring.full[x], 1);
    fence_mbar_init();
  }
  __syncthreads();
  const float over = 1.f / (float)n;
  const int64_t step = (int64_t)gridDim.x * shape.groups;
  int64_t row = (int64_t)blockIdx.x * shape.groups + group;
  after_previous();
  auto x_at = [&](int64_t i) { return static_cast<const T*>(a.X) + i * a.ldx; };
  auto g_at = [&](int64_t i) { return static_cast<const T*>(a.G) + i * a.ldg; };
  auto r_at = [&](int64_t i) { return static_cast<const T*>(a.R) + i * a.ldr; };
  auto fill = [&](int x, int64_t i) {
    if (i >= a.m) return;
    const T* p[3] = {x_at(i), g_at(i), a.R ? r_at(i) : nullptr};
    ring.fill(x, p, n, i + 1 == a.m);
  };
  if (t == 0)
    for (int x = 0; x < stages; ++x) fill(x, row + x * step);
  float w[CH], dw[SUMS ? CH : 1] = {}, db[SUMS ? CH : 1] = {};
#pragma unroll
  for (int i = 0; i < CH; ++i) w[i] = a.w && t + i * tpr < n ? to_f32(static_cast<const T*>(a.w)[t + i * tpr]) : 1.f;
  float mean_n = row < a.m ? a.mean_in[row] : 0.f, rstd_n = row < a.m ? a.rstd_in[row] : 0.f;
  for (; row < a.m; row += step) {
    const float mean = mean_n, rstd = rstd_n;
    const bool last = row + 1 == a.m;
    if (row + step < a.m) {
      mean_n = a.mean_in[row + step];
      rstd_n = a.rstd_in[row + step];
    }
    if (!ring.wait()) break;
    float u[CH], h[CH], res[CH];
    ring.load(0, x_at(row), t, tpr, n, last, u, mean);
    ring.load(1, g_at(row), t, tpr, n, last, h);
    if (a.R) ring.load(2, r_at(row), t, tpr, n, last, res);
    float2 s = make_float2(0.f, 0.f);
    // (beyond the row's end g is zero, and x mean: -mean rstd may be beyond fp32 where u is not)
#pragma unroll
    for (int i = 0; i < CH; ++i) {
      u[i] = (u[i] - mean) * rstd;
      if constexpr (SUMS) {
        dw[i] = fmaf(h[i], u[i], dw[i]);
        db[i] += h[i];
      }
      h[i] *= w[i];
      s.x += h[i];
      s.y = fmaf(h[i], u[i], s.y);
    }
    s = sum(s);
    if (t == 0) fill(ring.turn.s, row + stages * step);
    ring.turn.next();
    if (!a.DX) continue;
    const float c1 = s.x * over, c2 = s.y * over;
    T* out = static_cast<T*>(a.DX) + row * a.lddx;
#pragma unroll
    for (int i = 0; i < CH; ++i)
      if (t + i * tpr < n) out[t + i * tpr] = from_f32<T>(fmaf(fmaf(-u[i], c2, h[i] - c1), rstd, a.R ? res[i] : 0.f));
  }
  leave_rows<1>(ring, t == 0, group, tpr, row, a.m, step);
  if constexpr (SUMS)
    store_columns<T, 1, CH>(a, RowOf<T, 1, CH>(t, tpr, a.n), group, shape.groups, dw, db, reinterpret_cast<float*>(smem));
}

// Rows of at most 32 accesses of 16 bytes, without gaps between them: a row lies over `tpr` neighbouring lanes, an access
// each, and each warp has a ring of its own, of tiles of about 2 KB a matrix, several on their way at a time (with a row ahead in
// registers 1,000,000 x 32 float32 took 90 us).
constexpr int SHORT_THREADS = 512, SHORT_TILE = 2048, SHORT_BYTES = 192 * 1024;  // of a tile at most, of all rings

template <typename T, bool SUMS>
__global__ void __launch_bounds__(SHORT_THREADS, 1) norm_grad_short_kernel(const __grid_constant__ NormArgs a, const int tpr, const int rows,
                                                                          const int slot, const int stages) {
  constexpr int V = 16 / sizeof(T), P = V / 2, WARPS = SHORT_THREADS / 32;
  extern __shared__ __align__(128) unsigned char smem[];
  __shared__ __align__(8) uint64_t s_full[WARPS][MOST_STAGES];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, group = lane / tpr, t = lane % tpr, groups = 32 / tpr, accesses = (int)(a.n / V);
  const bool has = t < accesses;
  const int mats = a.R ? 3 : 2;
  const float over = 1.f / (float)a.n;
  unsigned char* at = smem + (size_t)warp * stages * mats * slot;
  uint64_t* full = s_full[warp];
  if (lane == 0) {
    for (int x = 0; x < stages; ++x) mbar_init(&full[x], 1);
    fence_mbar_init();
  }
  __syncwarp();
  after_previous();
  const int tiles = (int)((a.m + rows - 1) / rows), step = (int)gridDim.x * WARPS;  // (a tile has four rows at least)
  int tile = (int)blockIdx.x * WARPS + warp;
  auto fill = [&](int x, int i) {
    if (i >= tiles) return;
    const int64_t first = (int64_t)i * rows * a.n;
    const uint32_t bytes = (uint32_t)(min((int64_t)rows, a.m - (int64_t)i * rows) * accesses * 16);
    unsigned char* to = at + (size_t)x * mats * slot;
    mbar_arrive_expect_tx(&full[x], bytes * (uint32_t)mats);
    copy_row(to, static_cast<const T*>(a.X) + first, bytes, &full[x]);
    copy_row(to + slot, static_cast<const T*>(a.G) + first, bytes, &full[x]);
    if (a.R) copy_row(to + 2 * slot, static_cast<const T*>(a.R) + first, bytes, &full[x]);
  };
  if (lane == 0)
    for (int x = 0; x < stages; ++x) fill(x, tile + x * step);
  f2 dw[SUMS ? P : 1] = {}, db[SUMS ? P : 1] = {}, w[P];
  {
    Raw<T, V> raw;
    raw.zero();
    if (a.w && has) raw.load(static_cast<const T*>(a.w) + t * V);
    raw.pairs(w);
    if (!a.w) {
#pragma unroll
      for (int q = 0; q < P; ++q) w[q] = pack2(1.f, 1.f);
    }
  }
  RingTurn turn(stages);
  bool ok = true;
  // the statistics of a tile's rows (32 at most), a row a lane, a tile ahead
  float mean_n = 0.f, rstd_n = 0.f;
  auto fetch = [&](int i) {
    const int64_t r = (int64_t)i * rows + lane;
    const bool in = lane < rows && r < a.m;
    mean_n = in ? a.mean_in[r] : 0.f;
    rstd_n = in ? a.rstd_in[r] : 0.f;
  };
  fetch(tile);
  for (; tile < tiles; tile += step) {
    const int64_t row0 = (int64_t)tile * rows;
    const float mean_t = mean_n, rstd_t = rstd_n;
    fetch(tile + step);
    const int here = (int)min((int64_t)rows, a.m - row0);  // the tile's rows
    ok = __all_sync(FULL_MASK, ok && mbar_wait_bounded(&full[turn.s], turn.phase));
    if (!ok) {  // FXTX_ERR_TIMEOUT is raised
      if (lane == 0) drain(full, turn, tile, tiles, step);
      break;
    }
    const unsigned char* x_at = at + (size_t)turn.s * mats * slot + t * 16;
#pragma unroll 1
    for (int r0 = 0; r0 < here; r0 += 2 * groups) {
      f2 u[2][P], h[2][P], y[2][P];
      float scale[2], s1[2], s2[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * groups + group;
        const bool in = r < here;
        Raw<T, V> x, g, res;
        x.zero();
        g.zero();
        res.zero();
        float mean = __shfl_sync(FULL_MASK, mean_t, r & 31);
        scale[i] = __shfl_sync(FULL_MASK, rstd_t, r & 31);
        mean = in && has ? mean : 0.f;  // (beyond the row's end x and g are zero; -mean rstd may be beyond fp32 where u is not)
        if (in && has) {
          const unsigned char* p = x_at + r * accesses * 16;
          x.load(reinterpret_cast<const T*>(p));
          g.load(reinterpret_cast<const T*>(p + slot));
          if (a.R) res.load(reinterpret_cast<const T*>(p + 2 * slot));
        }
        x.pairs(u[i]);
        g.pairs(h[i]);
        res.pairs(y[i]);
        const f2 minus = pack2(-mean, -mean), sc = pack2(scale[i], scale[i]);
        f2 p1 = 0, p2 = 0;
#pragma unroll
        for (int q = 0; q < P; ++q) {
          u[i][q] = mul2(add2(u[i][q], minus), sc);
          if constexpr (SUMS) {
            dw[q] = fma2(h[i][q], u[i][q], dw[q]);
            db[q] = add2(db[q], h[i][q]);
          }
          h[i][q] = mul2(h[i][q], w[q]);
          p1 = add2(p1, h[i][q]);
          p2 = fma2(h[i][q], u[i][q], p2);
        }
        s1[i] = unpack2(p1).x + unpack2(p1).y;
        s2[i] = unpack2(p2).x + unpack2(p2).y;
      }
      if (!a.DX) continue;
      for (int o = tpr >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          s1[i] += shfl_xor(s1[i], o);
          s2[i] += shfl_xor(s2[i], o);
        }
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int r = r0 + i * groups + group;
        if (r >= here || !has) continue;
        const float c1 = -s1[i] * over, c2 = -s2[i] * over;
        const f2 d1 = pack2(c1, c1), d2 = pack2(c2, c2), sc = pack2(scale[i], scale[i]);
#pragma unroll
        for (int q = 0; q < P; ++q) y[i][q] = fma2(fma2(u[i][q], d2, add2(h[i][q], d1)), sc, y[i][q]);
        Raw<T, V>::store_pairs(static_cast<T*>(a.DX) + (row0 + r) * a.lddx + t * V, y[i]);
      }
    }
    __syncwarp();  // the tile has been read
    if (lane == 0) fill(turn.s, tile + stages * step);
    turn.next();
  }
  if constexpr (SUMS) {
    // a warp's by exchange, then warp after warp in shared memory: [2][V][tpr]
    __shared__ float cols[2 * V * 32];
    float x[V], y[V];
#pragma unroll
    for (int q = 0; q < P; ++q) {
      x[2 * q] = unpack2(dw[q]).x;
      x[2 * q + 1] = unpack2(dw[q]).y;
      y[2 * q] = unpack2(db[q]).x;
      y[2 * q + 1] = unpack2(db[q]).y;
    }
    for (int o = tpr; o < 32; o <<= 1)
#pragma unroll
      for (int e = 0; e < V; ++e) {
        x[e] += shfl_xor(x[e], o);
        y[e] += shfl_xor(y[e], o);
      }
    for (int z = 0; z < SHORT_THREADS / 32; ++z) {
      __syncthreads();
      if ((int)(threadIdx.x >> 5) != z || (int)(threadIdx.x & 31) >= tpr) continue;
#pragma unroll
      for (int e = 0; e < V; ++e) {
        float *p = cols + e * tpr + t, *q = p + V * tpr;
        *p = z > 0 ? *p + x[e] : x[e];
        *q = z > 0 ? *q + y[e] : y[e];
      }
    }
    __syncthreads();
    for (int j = threadIdx.x; j < a.n; j += SHORT_THREADS) {
      const float p = cols[j % V * tpr + j / V], q = cols[(V + j % V) * tpr + j / V];
      if (gridDim.x == 1) {
        if (a.DW) static_cast<T*>(a.DW)[j] = from_f32<T>(p);
        if (a.DB) static_cast<T*>(a.DB)[j] = from_f32<T>(q);
      } else {
        a.part[((int64_t)blockIdx.x * 2) * a.n + j] = p;
        a.part[((int64_t)blockIdx.x * 2 + 1) * a.n + j] = q;
      }
    }
  }
}

// dw and db from `parts` CTAs' sums, in order: 32 columns a CTA, 32 threads a column.
template <typename T>
__global__ void __launch_bounds__(1024) norm_join_kernel(const __grid_constant__ NormArgs a, int64_t parts) {
  __shared__ float part[32][33];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t j = (int64_t)blockIdx.x * 32 + x;
  float s = 0.f;
  after_previous();
  if (j < 2 * a.n) {
#pragma unroll 4
    for (int64_t p = y; p < parts; p += 32) s += a.part[p * 2 * a.n + j];
  }
  part[y][x] = s;
  __syncthreads();
  // a warp a column
  s = group_sum<32>(part[x][y]);
  const int64_t c = (int64_t)blockIdx.x * 32 + y;
  if (x != 0 || c >= 2 * a.n) return;
  T* to = static_cast<T*>(c < a.n ? a.DW : a.DB);
  if (to) to[c < a.n ? c : c - a.n] = from_f32<T>(s);
}

// A CTA's sums of two values, the same in every thread. (In doubles this took 5 us a row: two of them a cycle and SM.)
__device__ __forceinline__ float2 cta_sum(float x, float y, float2* red) {
  x = group_sum<32>(x);
  y = group_sum<32>(y);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = make_float2(x, y);
  __syncthreads();
  float2 s = make_float2(0.f, 0.f);
#pragma unroll
  for (int w = 0; w < LONG_THREADS / 32; ++w) {
    s.x += red[w].x;
    s.y += red[w].y;
  }
  return s;
}

// Rows of any length, one CTA a row at a time. A thread's sums leave fp32 after 16 accesses.
template <typename T, int V>
__global__ void __launch_bounds__(LONG_THREADS) norm_long_kernel(const __grid_constant__ NormArgs a) {
  __shared__ float2 red[LONG_THREADS / 32];
  after_previous();
  const int64_t accesses = a.n / V;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
    const T* x = static_cast<const T*>(a.X) + row * a.ldx;
    auto total = [&](auto term) {
      double s = 0.0;
      for (int64_t c0 = threadIdx.x; c0 < accesses; c0 += 16 * LONG_THREADS) {
        float p = 0.f;
#pragma unroll 4
        for (int i = 0; i < 16; ++i) {
          const int64_t c = c0 + (int64_t)i * LONG_THREADS;
          if (c >= accesses) break;
          Raw<T, V> raw;
          float v[V];
          raw.load(x + c * V);
          raw.values(v);
#pragma unroll
          for (int q = 0; q < V; ++q) p += term(v[q]);
        }
        s += p;
      }
      return cta_sum((float)s, 0.f, red).x;
    };
    const float mean = total([](float v) { return v; }) / (float)a.n;
    const float var = total([&](float v) { return (v - mean) * (v - mean); }) / (float)a.n;
    const float rstd = __frsqrt_rn(var + a.eps);
    if (threadIdx.x == 0) {
      if (a.mean) a.mean[row] = mean;
      if (a.rstd) a.rstd[row] = rstd;
    }
    T* out = static_cast<T*>(a.out) + row * a.ldo;
    for (int64_t c = threadIdx.x; c < accesses; c += LONG_THREADS) {
      Raw<T, V> raw;
      float v[V], y[V];
      raw.load(x + c * V);
      raw.values(v);
#pragma unroll
      for (int q = 0; q < V; ++q) v[q] = (v[q] - mean) * rstd;
      if (a.w) {
        raw.load(static_cast<const T*>(a.w) + c * V);
        raw.values(y);
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] *= y[q];
      }
      if (a.b) {
        raw.load(static_cast<const T*>(a.b) + c * V);
        raw.values(y);
#pragma unroll
        for (int q = 0; q < V; ++q) v[q] += y[q];
      }
      Raw<T, V>::store(out + c * V, v);
    }
  }
}

// The gradient of long rows, first pass: mean(h) and mean(h u) of each row.
template <typename T, int V>
__global__ void __launch_bounds__(LONG_THREADS) norm_long_means_kernel(const __grid_constant__ NormArgs a, float2* means) {
  __shared__ float2 red[LONG_THREADS / 32];
  after_previous();
  const int64_t accesses = a.n / V;
  for (int64_t row = blockIdx.x; row < a.m; row += gridDim.x) {
    const T *x = static_cast<const T*>(a.X) + row * a.ldx, *g = static_cast<const T*>(a.G) + row * a.ldg;
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
    double s = 0.0, t = 0.0;
    // four accesses of each on their way at a time
    constexpr int U = 4;
    for (int64_t c0 = threadIdx.x; c0 < accesses; c0 += U * LONG_THREADS) {
      Raw<T, V> xr[U], gr[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t c = c0 + (int64_t)i * LONG_THREADS;
        xr[i].zero();
        gr[i].zero();
        if (c < accesses) {
          xr[i].load(x + c * V);
          gr[i].load(g + c * V);
        }
      }
      float p = 0.f, o = 0.f;
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int64_t c = c0 + (int64_t)i * LONG_THREADS;
        float v[V], h[V], y[V];
        xr[i].values(v);
        gr[i].values(h);
        if (a.w && c < accesses) {
          Raw<T, V> raw;
          raw.load(static_cast<const T*>(a.w) + c * V);
          raw.values(y);
#pragma unroll
          for (int q = 0; q < V; ++q) h[q] *= y[q];
        }
        if (c >= accesses) continue;  // (-mean rstd may be beyond fp32 where u is not)
#pragma unroll
        for (int q = 0; q < V; ++q) {
          p += h[q];
          o = fmaf(h[q], (v[q] - mean) * rstd, o);
        }
      }
      s += p;
      t += o;
    }
    const float2 all = cta_sum((float)s, (float)t, red);
    if (threadIdx.x == 0) means[row] = make_float2(all.x / (float)a.n, all.y / (float)a.n);
  }
}

// Second pass: dx and the column sums; a thread keeps V columns and goes down `rows` rows.
template <typename T, int V>
__global__ void __launch_bounds__(256) norm_long_grad_kernel(const __grid_constant__ NormArgs a, const float2* means, int64_t slabs,
                                                             int64_t rows) {
  const int64_t slab = blockIdx.x % slabs, part = blockIdx.x / slabs, j = (slab * 256 + threadIdx.x) * V;
  after_previous();
  if (j >= a.n) return;
  Raw<T, V> raw;
  float w[V], dw[V] = {}, db[V] = {};
  if (a.w) {
    raw.load(static_cast<const T*>(a.w) + j);
    raw.values(w);
  }
  const int64_t end = min(a.m, (part + 1) * rows);
#pragma unroll 4
  for (int64_t row = part * rows; row < end; ++row) {
    float u[V], g[V], y[V];
    raw.load(static_cast<const T*>(a.X) + row * a.ldx + j);
    raw.values(u);
    raw.load(static_cast<const T*>(a.G) + row * a.ldg + j);
    raw.values(g);
    const float mean = a.mean_in[row], rstd = a.rstd_in[row];
#pragma unroll
    for (int q = 0; q < V; ++q) {
      u[q] = (u[q] - mean) * rstd;
      dw[q] = fmaf(g[q], u[q], dw[q]);
      db[q] += g[q];
    }
    if (!a.DX) continue;
    const float2 c = means[row];
    if (a.R) {
      raw.load(static_cast<const T*>(a.R) + row * a.ldr + j);
      raw.values(y);
    }
#pragma unroll
    for (int q = 0; q < V; ++q) {
      if (a.w) g[q] *= w[q];
      g[q] = (g[q] - c.x - u[q] * c.y) * rstd;
      if (a.R) g[q] += y[q];
    }
    Raw<T, V>::store(static_cast<T*>(a.DX) + row * a.lddx + j, g);
  }
  if (a.part) {
    float* p = a.part + part * 2 * a.n + j;
#pragma unroll
    for (int q = 0; q < V; ++q) {
      p[q] = dw[q];
      p[a.n + q] = db[q];
    }
  }
}

bool aligned(const void* p, int64_t ld, int size) { return p == nullptr || (((uintptr_t)p & 15u) == 0 && ld * size % 16 == 0); }

// Threads a row takes and rows a CTA has in work: `per` accesses a thread at most.
RowShape shape_of(int64_t accesses, int per, int threads) {
  RowShape s;
  const int64_t need = (accesses + per - 1) / per;
  if (need <= 32)
    while (s.tpr < need) s.tpr *= 2;
  else
    s.tpr = (int)((need + 31) / 32 * 32);
  s.groups = std::max(1, threads / s.tpr);
  return s;
}

// CTAs of a kernel that fit an SM, asked once for each of the row shapes (threads and shared memory go by tpr).
template <auto KERNEL>
int ctas_per_sm(int tpr, int threads, size_t smem) {
  static std::atomic<int> known[6 + 1024 / 32];
  int x = 0;
  if (tpr <= 32)
    while ((1 << x) < tpr) ++x;
  else
    x = 5 + tpr / 32 - 1;
  int b = known[x].load(std::memory_order_relaxed);
  if (b > 0) return b;
  if (cudaOccupancyMaxActiveBlocksPerMultiprocessor(&b, KERNEL, threads, smem) != cudaSuccess) cudaGetLastError();
  b = std::max(b, 1);
  known[x].store(b, std::memory_order_relaxed);
  return b;
}

template <typename T, int V, int CH, bool BIG>
cudaError_t launch_forward(const NormArgs& a, const RowShape& s, const DeviceInfo& dev, cudaStream_t st) {
  const int threads = (s.tpr * s.groups + 31) / 32 * 32;
  const int64_t fit = (int64_t)ctas_per_sm<norm_kernel<T, V, CH, BIG>>(s.tpr, threads, 0) * dev.sm_count;
  const int64_t grid = std::min<int64_t>((a.m + s.groups - 1) / s.groups, fit);
  return launch_kernel(norm_kernel<T, V, CH, BIG>, dim3((unsigned)grid), threads, 0, st, a, s);
}

template <typename T, int V, int CH>
cudaError_t forward_ch(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const RowShape s = shape_of(a.n / V, CH, FWD_THREADS);
  return s.tpr <= 32 ? launch_forward<T, V, CH, false>(a, s, dev, st) : launch_forward<T, V, CH, true>(a, s, dev, st);
}

// A ring's stages for rows of `bytes` and `mats` matrices; fewer than two: rows do not go that way.
int stages_of(const RowShape& s, int64_t bytes, int mats) {
  return (int)std::min<int64_t>(MOST_STAGES, RING_BYTES / (s.groups * mats * bytes));
}
// Rows of several warps, enough of them to keep the rings of all SMs full.
bool ring_rows(const RowShape& s, int64_t m, const DeviceInfo& dev) {
  return s.tpr > 32 && s.groups <= MOST_GROUPS && s.tpr <= RING_THREADS && m >= 4 * (int64_t)dev.sm_count * s.groups;
}

template <typename T, int CH>
cudaError_t launch_ring(const NormArgs& a, const RowShape& s, int stages, const DeviceInfo& dev, cudaStream_t st) {
  const size_t smem = (size_t)s.groups * stages * a.n * sizeof(T);
  const cudaError_t e = ensure_smem((const void*)norm_ring_kernel<T, CH>, smem);
  if (e != cudaSuccess) return e;
  return launch_kernel(norm_ring_kernel<T, CH>, dim3((unsigned)dev.sm_count), (unsigned)(s.tpr * s.groups), smem, st, a, s, stages);
}

// The shape of rows that come so: at most CH entries a thread, 64 threads at least; their slot in shared memory.
struct OddShape {
  RowShape s;
  int slot = 0, stages = 0;
};
bool odd_rows(const NormArgs& a, int size, int mats, const DeviceInfo& dev, OddShape& o) {
  if (a.n <= 128 || a.n > 16 * RING_THREADS) return false;
  for (const void* p : {a.X, a.G, a.R})
    if ((uintptr_t)p & 15u) return false;
  o.s.tpr = (int)std::max<int64_t>(64, ((a.n + 15) / 16 + 31) / 32 * 32);
  o.s.groups = RING_THREADS / o.s.tpr;
  o.slot = (int)((a.n * size + 15) / 16 * 16 + 32);
  o.stages = stages_of(o.s, o.slot, mats);
  return o.stages >= 2 && ring_rows(o.s, a.m, dev);
}

template <typename T, int CH>
cudaError_t launch_odd(const NormArgs& a, const OddShape& o, const DeviceInfo& dev, cudaStream_t st) {
  const size_t smem = (size_t)o.s.groups * o.stages * o.slot;
  const cudaError_t e = ensure_smem((const void*)norm_odd_kernel<T, CH>, smem + 1024);
  if (e != cudaSuccess) return e;
  return launch_kernel(norm_odd_kernel<T, CH>, dim3((unsigned)dev.sm_count), (unsigned)(o.s.tpr * o.s.groups), smem, st, a, o.s, o.slot, o.stages);
}

template <typename T, int V>
cudaError_t forward(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  constexpr int MOST = V == 1 ? 16 : 4;
  const int64_t accesses = a.n / V;
  if (accesses > (int64_t)MOST * 1024)
    return launch_kernel(norm_long_kernel<T, V>, dim3((unsigned)std::min<int64_t>(a.m, (int64_t)dev.sm_count * 4)), LONG_THREADS, 0,
                         st, a);
  if (accesses <= 32) return forward_ch<T, V, 1>(a, dev, st);
  if constexpr (V > 1) {
    const RowShape s = shape_of(accesses, MOST, RING_THREADS);
    const int stages = stages_of(s, a.n * (int64_t)sizeof(T), 1);
    if (stages >= 2 && ring_rows(s, a.m, dev)) return launch_ring<T, MOST>(a, s, stages, dev, st);
  } else {
    OddShape o;
    if (odd_rows(a, sizeof(T), 1, dev, o))
      return a.n <= 256 ? launch_odd<T, 4>(a, o, dev, st) : a.n <= 512 ? launch_odd<T, 8>(a, o, dev, st) : launch_odd<T, 16>(a, o, dev, st);
  }
  return forward_ch<T, V, MOST>(a, dev, st);
}

template <typename T, int V, int CH, bool BIG, bool SUMS>
fxtx_status_t launch_grad(NormArgs a, const RowShape& s, const DeviceInfo& dev, cudaStream_t st) {
  const int threads = (s.tpr * s.groups + 31) / 32 * 32;
  const size_t smem = SUMS ? (size_t)2 * CH * V * s.tpr * 4 : 0;
  // (its static shared memory counts too: 48 KB of dynamic alone do not fit without the attribute)
  cudaError_t e = ensure_smem((const void*)norm_grad_kernel<T, V, CH, BIG, SUMS>, smem + 1024);
  if (e != cudaSuccess) {
    cudaGetLastError();
    return FXTX_ERR_CUDA;
  }
  const int64_t fit = (int64_t)ctas_per_sm<norm_grad_kernel<T, V, CH, BIG, SUMS>>(s.tpr, threads, smem) * dev.sm_count;
  const int64_t grid = std::max<int64_t>(1, std::min<int64_t>((a.m + s.groups - 1) / s.groups, fit));  // (no rows: zero sums)
  if (SUMS && grid > 1) {
    const fxtx_status_t r = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)grid * 2 * a.n * 4, st);
    if (r != FXTX_OK) return r;
  }
  e = launch_kernel(norm_grad_kernel<T, V, CH, BIG, SUMS>, dim3((unsigned)grid), threads, smem, st, a, s);
  if (a.part) {
    if (e == cudaSuccess) e = launch_kernel(norm_join_kernel<T>, dim3((unsigned)((2 * a.n + 31) / 32)), 1024, 0, st, a, grid);
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

template <typename T, int V>
fxtx_status_t long_grad(NormArgs a, const DeviceInfo& dev, cudaStream_t st) {
  const bool sums = a.DW || a.DB;
  const int64_t slabs = (a.n / V + 255) / 256;
  const int64_t want = std::max<int64_t>(1, (int64_t)dev.sm_count * 4 / slabs);  // row ranges
  const int64_t rows = std::max<int64_t>(1, (a.m + want - 1) / want), parts = std::max<int64_t>(1, (a.m + rows - 1) / rows);
  const size_t mean_bytes = ((size_t)a.m * 8 + 255) / 256 * 256, part_bytes = sums ? (size_t)parts * 2 * a.n * 4 : 0;
  char* ws = nullptr;
  const fxtx_status_t r = alloc_pooled(reinterpret_cast<void**>(&ws), mean_bytes + part_bytes, st);
  if (r != FXTX_OK) return r;
  float2* means = reinterpret_cast<float2*>(ws);
  a.part = sums ? reinterpret_cast<float*>(ws + mean_bytes) : nullptr;
  cudaError_t e = cudaSuccess;
  if (a.DX && a.m > 0)
    e = launch_kernel(norm_long_means_kernel<T, V>, dim3((unsigned)std::min<int64_t>(a.m, (int64_t)dev.sm_count * 4)), LONG_THREADS, 0,
                      st, a, means);
  if (e == cudaSuccess)
    e = launch_kernel(norm_long_grad_kernel<T, V>, dim3((unsigned)(slabs * parts)), 256, 0, st, a, (const float2*)means, slabs, rows);
  if (e == cudaSuccess && sums) e = launch_kernel(norm_join_kernel<T>, dim3((unsigned)((2 * a.n + 31) / 32)), 1024, 0, st, a, parts);
  cudaFreeAsync(ws, st);
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

template <typename T, int CH, bool SUMS>
fxtx_status_t launch_grad_ring(NormArgs a, const RowShape& s, int stages, const DeviceInfo& dev, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T);
  const size_t sums = SUMS ? (size_t)2 * CH * V * s.tpr * 4 : 0;
  const size_t smem = std::max((size_t)s.groups * stages * (a.R ? 3 : 2) * a.n * sizeof(T), sums);
  cudaError_t e = ensure_smem((const void*)norm_grad_ring_kernel<T, CH, SUMS>, smem);
  if (SUMS && e == cudaSuccess) {
    const fxtx_status_t r = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)dev.sm_count * 2 * a.n * 4, st);
    if (r != FXTX_OK) return r;
  }
  if (e == cudaSuccess)
    e = launch_kernel(norm_grad_ring_kernel<T, CH, SUMS>, dim3((unsigned)dev.sm_count), (unsigned)(s.tpr * s.groups), smem, st, a, s, stages);
  if (a.part) {
    if (e == cudaSuccess) e = launch_kernel(norm_join_kernel<T>, dim3((unsigned)((2 * a.n + 31) / 32)), 1024, 0, st, a, (int64_t)dev.sm_count);
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

template <typename T, int CH, bool SUMS>
fxtx_status_t launch_grad_odd(NormArgs a, const OddShape& o, const DeviceInfo& dev, cudaStream_t st) {
  const size_t sums = SUMS ? (size_t)2 * CH * o.s.tpr * 4 : 0;
  const size_t smem = std::max((size_t)o.s.groups * o.stages * (a.R ? 3 : 2) * o.slot, sums);
  cudaError_t e = ensure_smem((const void*)norm_grad_odd_kernel<T, CH, SUMS>, smem + 1024);
  if (SUMS && e == cudaSuccess) {
    const fxtx_status_t r = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)dev.sm_count * 2 * a.n * 4, st);
    if (r != FXTX_OK) return r;
  }
  if (e == cudaSuccess)
    e = launch_kernel(norm_grad_odd_kernel<T, CH, SUMS>, dim3((unsigned)dev.sm_count), (unsigned)(o.s.tpr * o.s.groups), smem, st, a, o.s,
                      o.slot, o.stages);
  if (a.part) {
    if (e == cudaSuccess) e = launch_kernel(norm_join_kernel<T>, dim3((unsigned)((2 * a.n + 31) / 32)), 1024, 0, st, a, (int64_t)dev.sm_count);
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}
template <typename T, bool SUMS>
fxtx_status_t grad_odd(const NormArgs& a, const OddShape& o, const DeviceInfo& dev, cudaStream_t st) {
  return a.n <= 256   ? launch_grad_odd<T, 4, SUMS>(a, o, dev, st)
         : a.n <= 512 ? launch_grad_odd<T, 8, SUMS>(a, o, dev, st)
                      : launch_grad_odd<T, 16, SUMS>(a, o, dev, st);
}

template <typename T, bool SUMS>
fxtx_status_t launch_short(NormArgs a, const DeviceInfo& dev, cudaStream_t st) {
  const int accesses = (int)(a.n / (16 / (int)sizeof(T)));
  const RowShape s = shape_of(accesses, 1, 32);
  const int groups = 32 / s.tpr, rows = std::min(32, std::max(groups, SHORT_TILE / (accesses * 16) / groups * groups));
  const int slot = (rows * accesses * 16 + 127) / 128 * 128, each = SHORT_THREADS / 32 * (a.R ? 3 : 2) * slot;
  const int stages = std::min(MOST_STAGES, SHORT_BYTES / each);
  const size_t smem = (size_t)each * stages;
  cudaError_t e = ensure_smem((const void*)norm_grad_short_kernel<T, SUMS>, smem);
  const int64_t tiles = (a.m + rows - 1) / rows, grid = std::min<int64_t>((tiles + SHORT_THREADS / 32 - 1) / (SHORT_THREADS / 32), dev.sm_count);
  if (SUMS && e == cudaSuccess && grid > 1) {
    const fxtx_status_t r = alloc_pooled(reinterpret_cast<void**>(&a.part), (size_t)grid * 2 * a.n * 4, st);
    if (r != FXTX_OK) return r;
  }
  if (e == cudaSuccess) e = launch_kernel(norm_grad_short_kernel<T, SUMS>, dim3((unsigned)grid), SHORT_THREADS, smem, st, a, s.tpr, rows, slot, stages);
  if (a.part) {
    if (e == cudaSuccess) e = launch_kernel(norm_join_kernel<T>, dim3((unsigned)((2 * a.n + 31) / 32)), 1024, 0, st, a, grid);
    cudaFreeAsync(a.part, st);
  }
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

template <typename T, int V, int CH>
fxtx_status_t grad_ch(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const RowShape s = shape_of(a.n / V, CH, GRAD_THREADS);
  const bool sums = a.DW || a.DB;
  if (s.tpr <= 32)
    return sums ? launch_grad<T, V, CH, false, true>(a, s, dev, st) : launch_grad<T, V, CH, false, false>(a, s, dev, st);
  return sums ? launch_grad<T, V, CH, true, true>(a, s, dev, st) : launch_grad<T, V, CH, true, false>(a, s, dev, st);
}

template <typename T, int V>
fxtx_status_t grad(const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  constexpr int MOST = 16 / V;  // 16 entries a thread: with their sums, weights and the next row's they fill its registers
  const int64_t accesses = a.n / V;
  if (accesses > (int64_t)MOST * GRAD_THREADS) return long_grad<T, V>(a, dev, st);
  if constexpr (V > 1) {
    // (of fewer rows no warp has a second tile)
    if (accesses <= 32 && a.m * accesses >= (int64_t)dev.sm_count * SHORT_THREADS * 4 && a.ldx == a.n && a.ldg == a.n && (!a.R || a.ldr == a.n))
      return a.DW || a.DB ? launch_short<T, true>(a, dev, st) : launch_short<T, false>(a, dev, st);
    if (accesses <= 32) return grad_ch<T, V, 1>(a, dev, st);
    auto ring = [&](auto ch, fxtx_status_t& r) {
      constexpr int CH = decltype(ch)::value;
      const RowShape s = shape_of(accesses, CH, RING_THREADS);
      const int stages = stages_of(s, a.n * (int64_t)sizeof(T), a.R ? 3 : 2);
      if (stages < 2 || !ring_rows(s, a.m, dev)) return false;
      r = a.DW || a.DB ? launch_grad_ring<T, CH, true>(a, s, stages, dev, st) : launch_grad_ring<T, CH, false>(a, s, stages, dev, st);
      return true;
    };
    fxtx_status_t r;
    if (accesses <= 64 ? ring(std::integral_constant<int, 1>{}, r) : ring(std::integral_constant<int, MOST>{}, r)) return r;
  } else {
    if (accesses <= 32) return grad_ch<T, V, 1>(a, dev, st);
    OddShape o;
    if (odd_rows(a, sizeof(T), a.R ? 3 : 2, dev, o)) return a.DW || a.DB ? grad_odd<T, true>(a, o, dev, st) : grad_odd<T, false>(a, o, dev, st);
  }
  return grad_ch<T, V, MOST>(a, dev, st);
}

template <typename T>
fxtx_status_t run_t(const NormArgs& a, bool backward, const DeviceInfo& dev, cudaStream_t st) {
  constexpr int V = 16 / sizeof(T), S = sizeof(T);
  bool wide = a.n % V == 0 && aligned(a.X, a.ldx, S) && aligned(a.w, 0, S);
  if (backward) {
    wide = wide && aligned(a.G, a.ldg, S) && aligned(a.R, a.ldr, S) && aligned(a.DX, a.lddx, S);
    return wide ? grad<T, V>(a, dev, st) : grad<T, 1>(a, dev, st);
  }
  wide = wide && aligned(a.b, 0, S) && aligned(a.out, a.ldo, S);
  const cudaError_t e = wide ? forward<T, V>(a, dev, st) : forward<T, 1>(a, dev, st);
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

fxtx_status_t run(fxtx_type_t type, const NormArgs& a, bool backward, const DeviceInfo& dev, cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return run_t<float>(a, backward, dev, st);
    case FXTX_BF16: return run_t<__nv_bfloat16>(a, backward, dev, st);
    default: return run_t<__half>(a, backward, dev, st);
  }
}

}  // namespace

fxtx_status_t run_norm(fxtx_type_t type, const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  return run(type, a, false, dev, st);
}
fxtx_status_t run_norm_grad(fxtx_type_t type, const NormArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  return run(type, a, true, dev, st);
}

}  // namespace fxtx
