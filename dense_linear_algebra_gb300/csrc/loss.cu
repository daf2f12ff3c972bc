// loss.cu — softmax cross entropy on a linear layer's outputs, and its gradient, without the outputs being kept:
//     z = X W + b,  lse_i = log sum_j exp z_ij,  loss_i = lse_i - z_i,label
//     D_ij = g_i (exp(z_ij - lse_i) - [j = label_i]),  dX = D W^T,  dW = X^T D,  db = the column sums of D
//
// Bound: the tensor cores, 2 m n k operations forward and 6 m n k backward (z is formed again), or with few rows the
// stream of W. 8192 x 2048, 65,536 classes in bfloat16: 1.10 ms (2,000 TFLOP/s) and 3.64 ms (1,815; at the power limit 1.29 and
// 4.1 ms); one row of 4096, 32,000 classes 53 us (5.0 TB/s).
//
// Forward: one product whose epilogue reduces each row of a tile to its largest entry and its sum of exponentials; a
// second kernel joins a row's parts. Nothing of the size of z is written.
//
// Backward: W in pieces of the classes and X in slabs of rows, so that D of one piece and slab takes kCap bytes at most.
// Per piece and slab three products: z again, whose epilogue writes D as an operand of the others (of the layer's type,
// of float32 as three bfloat16 planes) and its column sums; D W^T, added up over the pieces in fp32; X^T D, over the slabs.
//
// D of a 16-bit type is rounded to it, as linear_grad's is: dX and dW are then 2.4e-3 off in bfloat16 (2-norm, relative; 1.7e-3, the
// result's own rounding, with D in fp32). As the sum of two 16-bit terms it would take dX and dW twice, 1.2 of 3.64 ms more.
//
// float16 has nothing below 6e-8, where a mean's gradient over many classes lies: D is held multiplied by the power of
// two that brings the largest |g| of a row with a label to 2^14 .. 2^15, which the last of the sums takes back. What is lost is below
// 2^-39 of that |g| (below 2^-29 of it, digits are).
//
// At most 64 features and classes: thin_loss.cu, and thin_loss_f32.cu. Few rows: z is written out in fp32, its statistics or D
// formed by kernels of their own, and the products are those of few rows.
#include <algorithm>

#include "act.cuh"
#include "common.cuh"
#include "host.h"
#include "kernels.h"
#include "loss.h"

namespace fxtx {
namespace {

// Workspace for D (or few float32 rows' planes of W), and for each other array that goes in pieces: the pool keeps 1 GB between calls.
constexpr int64_t kCap = (int64_t)512 << 20, kSmallCap = (int64_t)256 << 20;
constexpr int64_t kRows = 16384;  // of a slab, where the classes leave the choice

fxtx_status_t status_of(cudaError_t e) {
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

// A row's statistics from its parts, and its loss: RX rows a CTA, 256 / RX threads a row, 8 parts on their way at a time.
template <int RX>
__global__ void __launch_bounds__(256) loss_join_kernel(const float2* stats, int64_t parts, int64_t rows, const float* target,
                                                        const void* labels, bool labels64, int64_t count, float* loss, float* lse) {
  constexpr int RY = 256 / RX;
  __shared__ float2 part[RY][RX];
  const int x = threadIdx.x % RX, y = threadIdx.x / RX;
  const int64_t i = (int64_t)blockIdx.x * RX + x;
  float top = -INFINITY, sum = 0.f;
  auto add = [&](const float2* s, int n) {
    float most = top;
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) most = fmaxf(most, s[q].x);
    const float from = most == -INFINITY ? 0.f : most;
    sum *= expf(top - from);
#pragma unroll
    for (int q = 0; q < 8; ++q)
      if (q < n) sum += s[q].y * expf(s[q].x - from);
    top = most;
  };
  after_previous();
  if (i < rows) {
    for (int64_t p = y; p < parts; p += 8 * RY) {
      float2 s[8];
#pragma unroll
      for (int q = 0; q < 8; ++q) s[q] = p + q * RY < parts ? stats[(p + q * RY) * rows + i] : make_float2(-INFINITY, 0.f);
      add(s, 8);
    }
  }
  part[y][x] = make_float2(top, sum);
  // a row's threads two by two
  for (int o = RY / 2; o > 0; o >>= 1) {
    __syncthreads();
    if (y >= o) continue;
    add(&part[y + o][x], 1);
    part[y][x] = make_float2(top, sum);
  }
  if (y != 0 || i >= rows) return;
  const float from = top == -INFINITY ? 0.f : top, rest = logf(sum);
  if (lse) lse[i] = from + rest;
  if (loss) loss[i] = label_at(labels, labels64, i, count) >= 0 ? (from - target[i]) + rest : 0.f;
}

cudaError_t launch_join(const float2* stats, int64_t parts, int64_t rows, const float* target, const void* labels, bool labels64,
                        int64_t count, float* loss, float* lse, const DeviceInfo& dev, cudaStream_t st) {
  // few rows: a CTA each
  const int rx = rows < 8 * (int64_t)dev.sm_count ? 1 : 8;
  const dim3 grid((unsigned)((rows + rx - 1) / rx));
  return rx == 1 ? launch_kernel(loss_join_kernel<1>, grid, 256, 0, st, stats, parts, rows, target, labels, labels64, count, loss, lse)
                 : launch_kernel(loss_join_kernel<8>, grid, 256, 0, st, stats, parts, rows, target, labels, labels64, count, loss, lse);
}

constexpr int SEG = 1024;  // of a row that a CTA reduces
// Rows whose logits are written out, at most. Of 16 bits (us, written out and in tiles; bfloat16):
//   loss       2048 x 32,000  1 row 32 and 45, 16 rows 33 and 46, 32 rows 36 and 35, 64 rows 41 and 36; 8192 x 4000  1 row 15 and 47, 64 rows 18
//              and 30; 1024 x 8000  16 rows 12 and 13, 32 rows 13 and 13; 512 x 50,000  1 row 23 and 20; 4096 x 131,072  1 row 263 and 245
//   gradient   2048 x 32,000  1 row 126 and 135, 4 rows 127 and 130, 16 rows 132 and 130; 8192 x 4000  4 rows 65 and 113, 16 rows 72 and 89;
//              512 x 50,000  4 rows 79 and 77, 16 rows 88 and 77
// and the loss of float32: 2048 x 32,000  24 rows 199 and 211, 128 rows 212 and 214, 256 rows 290 and 289; 8192 x 4000  128 rows 113 and 208;
// 512 x 50,000  24 rows 89 and 92, 128 rows 108 and 92.
constexpr int kFewLogits = 16, kFewLogitsGrad = 4, kFewLogitsF32 = 128;
// The rows that few_logits leaves to the gradient's way, at most: float32's are those of the CUDA cores.
constexpr int kSlopeRows = std::max({kFewLogitsGrad, kFewByRow, kFewByColumn});

// Few rows' logits in memory: `parts` parts of X W to be added, [part][row][class], and the biases.
struct FewLogits {
  const float* z;
  int64_t rows, k;
  int parts;
  const void* bias;
};
template <typename T>
__device__ __forceinline__ float logit(const FewLogits& f, int64_t i, int64_t j) {
  float z = 0.f;
  for (int p = 0; p < f.parts; ++p) z += f.z[(p * f.rows + i) * f.k + j];
  return f.bias ? z + to_f32(static_cast<const T*>(f.bias)[j]) : z;
}

// Their statistics: part s of row i is columns SEG s and on.
template <typename T>
__global__ void __launch_bounds__(256) row_stats_kernel(const FewLogits f, int64_t segs, float2* stats, float* target, const void* labels,
                                                        bool labels64) {
  __shared__ float2 part[8];
  const int64_t i = blockIdx.x / segs, s = blockIdx.x % segs, j0 = s * SEG, end = min(f.k, j0 + SEG);
  after_previous();
  float v[SEG / 256], top = -INFINITY, sum = 0.f;
#pragma unroll
  for (int q = 0; q < SEG / 256; ++q) {
    const int64_t j = j0 + q * 256 + threadIdx.x;
    v[q] = j < end ? logit<T>(f, i, j) : -INFINITY;
    top = fmaxf(top, v[q]);
  }
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, shfl_xor(top, o));
  const float from = top == -INFINITY ? 0.f : top;
#pragma unroll
  for (int q = 0; q < SEG / 256; ++q) sum += expf(v[q] - from);
  sum = group_sum<32>(sum);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = make_float2(top, sum);
  __syncthreads();
  if (threadIdx.x != 0) return;
  float most = -INFINITY, all = 0.f;
  for (int w = 0; w < 8; ++w) most = fmaxf(most, part[w].x);
  const float base = most == -INFINITY ? 0.f : most;
  for (int w = 0; w < 8; ++w) all += part[w].y * expf(part[w].x - base);
  stats[s * f.rows + i] = make_float2(most, all);
  const int64_t label = label_at(labels, labels64, i, f.k);
  if (label >= j0 && label < end) target[i] = logit<T>(f, i, label);
}

// Their D and db: a thread takes a class and goes down the rows.
template <typename T>
__global__ void __launch_bounds__(256) row_slope_kernel(const FewLogits f, const void* labels, bool labels64, const float* lse, const float* g,
                                                        float gain, const float* scales, T* D, int64_t ldd, T* db) {
  struct Row {
    float lse, g;
    int64_t label;
  };
  __shared__ Row rows[kSlopeRows];
  after_previous();
  const float up = scales ? scales[0] : 1.f;
  for (int i = threadIdx.x; i < f.rows; i += 256) {
    Row r;
    r.label = label_at(labels, labels64, i, f.k);
    r.lse = lse[i];
    r.g = g ? gain * g[i] : gain;
    rows[i] = r;
  }
  __syncthreads();
  const int64_t j = (int64_t)blockIdx.x * 256 + threadIdx.x;
  if (j >= f.k) return;
  float sum = 0.f;
#pragma unroll 4
  for (int i = 0; i < f.rows; ++i) {
    const Row r = rows[i];
    float d = 0.f;
    if (r.label >= 0) {
      const float w = r.g * up;
      d = w * expf(logit<T>(f, i, j) - r.lse);
      if (j == r.label) d -= w;
    }
    D[i * ldd + j] = from_f32<T>(d);
    sum += d;
  }
  if (db) db[j] = from_f32<T>(scales ? sum * scales[1] : sum);
}

// The powers of two that float16's D is held at, from the largest |g| of a row that has a label (as its bits: magnitudes order as
// integers do, a NaN above all).
__device__ __forceinline__ void set_scales(uint32_t most, float gain, float* scales) {
  const float top = __uint_as_float(most) * fabsf(gain);
  int e = 14;
  if (top > 0.f && top <= 3.4e38f) e = min(max(ilogbf(top), -100), 120);
  scales[0] = scalbnf(1.f, 14 - e);
  scales[1] = scalbnf(1.f, e - 14);
}

// A CTA's part of the rows; a single one's is all. (1,000,000 x 32, 10 classes: 54 us in all; one CTA for all weights 116.)
__global__ void __launch_bounds__(1024) largest_kernel(const void* labels, bool labels64, int64_t count, const float* g, int64_t m,
                                                       float gain, float* scales) {
  __shared__ uint32_t warps[32];
  after_previous();
  uint32_t most = 0;
  const int64_t step = (int64_t)gridDim.x * 1024;
#pragma unroll 4
  for (int64_t i = (int64_t)blockIdx.x * 1024 + threadIdx.x; i < m; i += step) {
    const uint32_t bits = __float_as_uint(g[i]) & 0x7fffffffu;
    most = max(most, label_at(labels, labels64, i, count) >= 0 ? bits : 0u);
  }
  most = __reduce_max_sync(FULL_MASK, most);
  if ((threadIdx.x & 31) == 0) warps[threadIdx.x >> 5] = most;
  __syncthreads();
  if (threadIdx.x != 0) return;
  for (int w = 1; w < 32; ++w) most = max(most, warps[w]);
  if (gridDim.x == 1) set_scales(most, gain, scales);
  else reinterpret_cast<uint32_t*>(scales)[2 + blockIdx.x] = most;
}

// The same from `parts` CTAs' parts; without any (no weights) from 1.
__global__ void __launch_bounds__(32) scales_kernel(int parts, float gain, float* scales) {
  after_previous();
  uint32_t most = parts ? 0u : __float_as_uint(1.f);
  for (int i = threadIdx.x; i < parts; i += 32) most = max(most, reinterpret_cast<const uint32_t*>(scales)[2 + i]);
  most = __reduce_max_sync(FULL_MASK, most);
  if (threadIdx.x == 0) set_scales(most, gain, scales);
}

// db from the column sums of D: 32 columns a CTA, 8 threads a column, in order; over the slabs through `keep`.
template <typename T>
__global__ void __launch_bounds__(256) db_join_kernel(const float* sums, int64_t parts, int64_t cols, const float* in, float* keep,
                                                      const float* scales, T* db) {
  __shared__ float part[8][32];
  const int x = threadIdx.x & 31, y = threadIdx.x >> 5;
  const int64_t j = (int64_t)blockIdx.x * 32 + x;
  float s = 0.f;
  after_previous();
  if (j < cols) {
#pragma unroll 4
    for (int64_t p = y; p < parts; p += 8) s += sums[p * cols + j];
  }
  part[y][x] = s;
  __syncthreads();
  if (y != 0 || j >= cols) return;
  for (int i = 1; i < 8; ++i) s += part[i][x];
  if (in) s += in[j];
  if (keep) keep[j] = s;
  else db[j] = from_f32<T>(scales ? s * scales[1] : s);
}

size_t up(int64_t bytes) { return (size_t)((bytes + 255) / 256 * 256); }
int64_t floor256(int64_t x) { return std::max<int64_t>(256, x / 256 * 256); }

// A workspace cut into arrays: sizes first, then addresses.
struct Cut {
  char* base = nullptr;
  size_t bytes = 0;
  char* take(int64_t n) {
    char* p = base ? base + bytes : nullptr;
    bytes += up(n);
    return n ? p : nullptr;
  }
};

// `rows` rows of a row-major matrix from row r on, `cols` columns from column c on, as an operand; packed to `at` if it must be.
struct Part {
  Operand o;
  PackArgs pack;
  bool packed = false;
  Planes planes;
};
const char* entry(const void* p, int64_t ld, int64_t r, int64_t c, int size) { return static_cast<const char*>(p) + (r * ld + c) * size; }

Part part_of(fxtx_type_t type, const void* p, int64_t ld, int64_t r, int64_t rows, int64_t c, int64_t cols, char* at) {
  Part x;
  x.o.p = entry(p, ld, r, c, type_size(type));
  x.o.ld = ld;
  size_t need = 0;
  x.planes = planes_of(x.o, type, rows, cols, at, &need);  // (K-major: rows x cols in memory)
  if (need) {
    x.packed = true;
    x.pack.src = x.o.p;
    x.pack.rows = rows;
    x.pack.cols = cols;
    x.pack.ld = ld;
    x.pack.dst = at;
    x.pack.pitch = x.planes.pitch;
    x.pack.plane_stride = x.planes.plane_stride;
    x.o.p = at;
    x.o.ld = x.planes.pitch;
    x.o.plane_stride = type == FXTX_F32 ? x.planes.plane_stride : 0;
  }
  return x;
}
// The same matrix as an operand whose kk runs along its rows, or along its columns.
Planes as(const Part& x, bool mn_major) {
  Planes p = x.planes;
  p.mn_major = mn_major;
  return p;
}

// Of an operand that has to be packed (float32, or 16 bits that the tensor copies cannot read where they lie): the bytes
// a row (or column) of it takes; else 0.
int64_t packed_bytes(fxtx_type_t type, const void* p, int64_t ld, int64_t entries) {
  Operand o;
  o.p = p;
  o.ld = ld;
  if (type != FXTX_F32 && copyable(o)) return 0;
  return (entries + 7) / 8 * 8 * (type == FXTX_F32 ? 6 : 2);
}

// The classes of W from c on: rows of a matrix stored by columns, else columns.
Part classes_of(const LayerArgs& l, int64_t c, int64_t n, char* at) {
  return l.w_trans ? part_of(l.type, l.W, l.ldw, c, n, 0, l.n, at) : part_of(l.type, l.W, l.ldw, 0, l.n, c, n, at);
}

// An even division into pieces of at most `most` (a multiple of 256).
int64_t piece_of(int64_t n, int64_t most) {
  if (n <= most) return n;
  const int64_t pieces = (n + most - 1) / most;
  return ((n + pieces - 1) / pieces + 255) / 256 * 256;
}

const void* bias_at(const LayerArgs& l, int64_t c) {
  return l.e.bias ? static_cast<const char*>(l.e.bias) + c * type_size(l.type) : nullptr;
}

const void* labels_at(const LossArgs& a, int64_t r) { return static_cast<const char*>(a.labels) + r * (a.labels64 ? 8 : 4); }

// W's planes as the linear layer takes them, all of float32's classes at once.
int64_t planes_bytes(const LayerArgs& l) { return 6 * l.k * ((l.n + 7) / 8 * 8); }

// Whether a call's logits are written out, in fp32: few rows', which the product kernels of few rows take (W is read once with
// no row of the tile wasted), or for float32 the CUDA cores. The gradient of float32 rows that those do not take forms
// W's planes once for all of its products instead, and so does that of rows whose dX needs planes that go in pieces only.
bool few_logits(const LayerArgs& l, const LossArgs* grad) {
  if (l.m * l.k * 4 > kSmallCap) return false;
  if (l.type != FXTX_F32) return l.m <= (grad ? kFewLogitsGrad : kFewLogits) && packed_bytes(l.type, l.W, l.ldw, l.n) == 0;
  if (!grad) return l.m <= kFewLogitsF32;
  return few_rows(l.type, l.m, l.w_trans) && (!grad->DX || few_rows(l.type, l.m, !l.w_trans) || planes_bytes(l) <= kCap);
}

// Few rows as an operand, in a workspace of its own where they have to be copied.
struct FewRows {
  Part x;
  char* at = nullptr;
};
fxtx_status_t few_operand(const LayerArgs& l, FewRows* f, const DeviceInfo& dev, cudaStream_t st) {
  const fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&f->at), (size_t)(l.m * packed_bytes(l.type, l.X, l.ldx, l.n)), st);
  if (s != FXTX_OK) return s;
  f->x = part_of(l.type, l.X, l.ldx, 0, l.m, 0, l.n, f->at);
  return f->x.packed ? status_of(launch_prepare(l.type, nullptr, &f->x.pack, 1, dev.sm_count, st)) : FXTX_OK;
}

PlanesProduct logits_product(const LayerArgs& l, const Part& x) {
  const Part w = classes_of(l, 0, l.k, nullptr);
  PlanesProduct q;
  q.M = l.m;
  q.N = l.k;
  q.K = l.n;
  q.A = as(x, false);
  q.B = as(w, !l.w_trans);
  return q;
}

// X W of few rows to z; its biases are left to the kernels that read it. Of float32 W goes in pieces of the classes where its planes
// would take more than kCap (128 x 4096, 131,072 classes: 3.2 GB at once 1,664 us, in pieces 1,556).
fxtx_status_t run_logits(const LayerArgs& l, const Part& x, float* z, const DeviceInfo& dev, cudaStream_t st) {
  if (l.type != FXTX_F32) return run_raw(l.type, logits_product(l, x), z, dev, st);
  const int64_t row = (l.n + 7) / 8 * 8 * 6, most = few_rows(l.type, l.m, l.w_trans) ? l.k : floor256(kCap / row);
  const int64_t Vp = piece_of(l.k, most);
  LayerArgs z_of = l;
  z_of.e = Epilogue{};
  z_of.e.ldo = l.k;
  fxtx_status_t s = FXTX_OK;
  for (int64_t v = 0; v < l.k && s == FXTX_OK; v += Vp) {
    z_of.k = std::min(Vp, l.k - v);
    z_of.W = l.w_trans ? entry(l.W, l.ldw, v, 0, 4) : entry(l.W, l.ldw, 0, v, 4);
    z_of.e.out = z + v;
    s = run_linear(z_of, dev, st);
  }
  return s;
}

template <typename T>
fxtx_status_t few_loss(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  FewRows x;
  fxtx_status_t s = l.type == FXTX_F32 ? FXTX_OK : few_operand(l, &x, dev, st);
  const int64_t segs = (l.k + SEG - 1) / SEG, parts = l.type == FXTX_F32 ? 1 : raw_parts(logits_product(l, x.x), dev);
  const size_t z_bytes = up(parts * l.m * l.k * 4), stat_bytes = up(segs * l.m * 8);
  char* ws = nullptr;
  if (s == FXTX_OK) s = alloc_pooled(reinterpret_cast<void**>(&ws), z_bytes + stat_bytes + up(l.m * 4), st);
  float *z = reinterpret_cast<float*>(ws), *target = reinterpret_cast<float*>(ws + z_bytes + stat_bytes);
  float2* stats = reinterpret_cast<float2*>(ws + z_bytes);
  if (s == FXTX_OK) s = run_logits(l, x.x, z, dev, st);
  if (s == FXTX_OK)
    s = status_of(launch_kernel(row_stats_kernel<T>, dim3((unsigned)(l.m * segs)), 256, 0, st, FewLogits{z, l.m, l.k, (int)parts, l.e.bias},
                                segs, stats, target, a.labels, a.labels64));
  if (s == FXTX_OK) s = status_of(launch_join(stats, segs, l.m, target, a.labels, a.labels64, l.k, a.loss, a.lse, dev, st));
  if (ws) cudaFreeAsync(ws, st);
  if (x.at) cudaFreeAsync(x.at, st);
  return s;
}

template <typename T>
fxtx_status_t few_grad(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  const bool f32 = l.type == FXTX_F32;
  FewRows x;
  fxtx_status_t s = f32 ? FXTX_OK : few_operand(l, &x, dev, st);
  const int64_t parts = f32 ? 1 : raw_parts(logits_product(l, x.x), dev), pitch = (l.k + 7) / 8 * 8;
  const size_t z_bytes = up(parts * l.m * l.k * 4), d_bytes = up(l.m * pitch * type_size(l.type));
  char* ws = nullptr;
  if (s == FXTX_OK) s = alloc_pooled(reinterpret_cast<void**>(&ws), z_bytes + d_bytes + kScaleBytes, st);
  float* z = reinterpret_cast<float*>(ws);
  T* D = reinterpret_cast<T*>(ws + z_bytes);
  float* scales = l.type == FXTX_F16 ? reinterpret_cast<float*>(ws + z_bytes + d_bytes) : nullptr;
  if (s == FXTX_OK && scales) s = status_of(launch_scales(a, l.m, l.k, scales, st));
  if (s == FXTX_OK) s = run_logits(l, x.x, z, dev, st);
  if (s == FXTX_OK)
    s = status_of(launch_kernel(row_slope_kernel<T>, dim3((unsigned)((l.k + 255) / 256)), 256, 0, st,
                                FewLogits{z, l.m, l.k, (int)parts, l.e.bias}, a.labels, a.labels64, a.lse_in, a.g, a.gain, scales, D, pitch,
                                static_cast<T*>(a.DB)));
  if (f32 && s == FXTX_OK && (a.DX || a.DW)) {
    GradArgs g;
    g.G = D;
    g.ldg = pitch;
    g.DX = a.DX;
    g.lddx = a.lddx;
    g.DW = a.DW;
    g.lddw = a.lddw;
    s = run_grad(l, g, dev, st);
  }
  if (!f32) {
    const Part w = classes_of(l, 0, l.k, nullptr);
    Planes d;
    d.p = D;
    d.rows = l.m;
    d.cols = l.k;
    d.pitch = pitch;
    d.plane_stride = l.m * pitch;
    ModeArgs<3> m;
    m.scales = scales;
    if (s == FXTX_OK && a.DX) {
      PlanesProduct t;
      t.M = l.m;
      t.N = l.n;
      t.K = l.k;
      t.A = d;
      t.B = as(w, l.w_trans);
      const int64_t dx_parts = raw_parts(t, dev);
      float* sums = nullptr;
      s = alloc_pooled(reinterpret_cast<void**>(&sums), (size_t)(dx_parts * l.m * l.n * 4), st);
      if (s == FXTX_OK) s = run_raw(l.type, t, sums, dev, st);
      if (s == FXTX_OK) s = join_sums(l.type, m, a.DX, a.lddx, l.m, l.n, dx_parts, sums, dev, st);
      if (sums) cudaFreeAsync(sums, st);
    }
    if (s == FXTX_OK && a.DW) {
      Planes dm = d, xm = as(x.x, true);
      dm.mn_major = true;
      PlanesProduct t;
      t.M = l.w_trans ? l.k : l.n;
      t.N = l.w_trans ? l.n : l.k;
      t.K = l.m;
      t.A = l.w_trans ? dm : xm;
      t.B = l.w_trans ? xm : dm;
      t.e.out = a.DW;
      t.e.ldo = a.lddw;
      s = run_sum(l.type, t, m, dev, st);
    }
  }
  if (ws) cudaFreeAsync(ws, st);
  if (x.at) cudaFreeAsync(x.at, st);
  return s;
}

}  // namespace

cudaError_t launch_scales(const LossArgs& a, int64_t m, int64_t k, float* scales, cudaStream_t st) {
  int parts = 0;
  if (a.g) {
    parts = (int)std::min<int64_t>(kScaleParts, (m + 8191) / 8192);  // (of 8 rows a thread)
    const cudaError_t e = launch_kernel(largest_kernel, dim3((unsigned)parts), 1024, 0, st, a.labels, a.labels64, k, a.g, m, a.gain, scales);
    if (e != cudaSuccess || parts == 1) return e;
  }
  return launch_kernel(scales_kernel, dim3(1), 32, 0, st, parts, a.gain, scales);
}

fxtx_status_t run_loss(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  if (few_logits(l, nullptr)) switch (l.type) {
      case FXTX_F32: return few_loss<float>(l, a, dev, st);
      case FXTX_BF16: return few_loss<__nv_bfloat16>(l, a, dev, st);
      default: return few_loss<__half>(l, a, dev, st);
    }
  // W's classes go in pieces where they have to be packed, X's rows also where the parts' statistics would take more
  const int64_t w_row = packed_bytes(l.type, l.W, l.ldw, l.n), x_row = packed_bytes(l.type, l.X, l.ldx, l.n);
  const int64_t Vp = piece_of(l.k, w_row ? floor256(kSmallCap / w_row) : l.k), pieces = (l.k + Vp - 1) / Vp;
  const int64_t parts_most = (Vp + 31) / 32 + 8;  // of a piece
  int64_t most = floor256(kSmallCap / (8 * parts_most * pieces));
  if (x_row) most = std::min(most, floor256(kSmallCap / x_row));
  const int64_t mc = piece_of(l.m, most);

  Cut c;
  char *ws = nullptr, *w_at = nullptr, *x_at = nullptr;
  float2* stats = nullptr;
  float* target = nullptr;
  for (int pass = 0; pass < 2; ++pass) {
    // (the pitch of W stored by rows runs over the classes)
    w_at = c.take(w_row ? (l.w_trans ? Vp * w_row : l.n * ((Vp + 7) / 8 * 8) * (l.type == FXTX_F32 ? 6 : 2)) : 0);
    x_at = c.take(mc * x_row);
    stats = reinterpret_cast<float2*>(c.take(parts_most * pieces * mc * 8));
    target = reinterpret_cast<float*>(c.take(mc * 4));
    if (pass == 0) {
      const fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&ws), c.bytes, st);
      if (s != FXTX_OK) return s;
      c.base = ws;
      c.bytes = 0;
    }
  }
  fxtx_status_t s = FXTX_OK;
  for (int64_t r = 0; r < l.m && s == FXTX_OK; r += mc) {
    const int64_t rows = std::min(mc, l.m - r);
    const Part x = part_of(l.type, l.X, l.ldx, r, rows, 0, l.n, x_at);
    int64_t parts = 0;
    for (int64_t v = 0; v < l.k && s == FXTX_OK; v += Vp) {
      const int64_t n = std::min(Vp, l.k - v);
      const Part w = classes_of(l, v, n, w_at);
      PackArgs packs[2];
      int count = 0;
      if (x.packed && v == 0) packs[count++] = x.pack;
      if (w.packed && (pieces > 1 || r == 0)) packs[count++] = w.pack;
      if (count) s = status_of(launch_prepare(l.type, nullptr, packs, count, dev.sm_count, st));
      PlanesProduct q;
      q.M = rows;
      q.N = n;
      q.K = l.n;
      q.A = as(x, false);
      q.B = as(w, !l.w_trans);
      q.e.bias = bias_at(l, v);
      ModeArgs<1> m;
      m.labels = labels_at(a, r);
      m.labels64 = a.labels64;
      m.count = l.k;
      m.col0 = v;
      m.stats = stats + parts * rows;
      m.target = target;
      if (s == FXTX_OK) s = run_stats(l.type, q, m, dev, st);
      parts += stat_parts(l.type, q, dev);
    }
    if (s == FXTX_OK)
      s = status_of(launch_join(stats, parts, rows, target, labels_at(a, r), a.labels64, l.k, a.loss ? a.loss + r : nullptr,
                                a.lse ? a.lse + r : nullptr, dev, st));
  }
  cudaFreeAsync(ws, st);
  return s;
}

fxtx_status_t run_loss_grad(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st) {
  if (few_logits(l, &a)) switch (l.type) {
      case FXTX_F32: return few_grad<float>(l, a, dev, st);
      case FXTX_BF16: return few_grad<__nv_bfloat16>(l, a, dev, st);
      default: return few_grad<__half>(l, a, dev, st);
    }
  const bool f32 = l.type == FXTX_F32;
  const int size = type_size(l.type), d_size = f32 ? 6 : 2;
  const int64_t w_row = packed_bytes(l.type, l.W, l.ldw, l.n), x_row = packed_bytes(l.type, l.X, l.ldx, l.n);
  // slabs of rows and pieces of classes
  int64_t mc = std::min(l.m, kRows);
  int64_t v_most = floor256(kCap / (d_size * mc));
  if (w_row) v_most = std::min(v_most, floor256(kSmallCap / w_row));
  const int64_t Vp = piece_of(l.k, v_most);
  int64_t m_most = floor256(kCap / (d_size * ((Vp + 7) / 8 * 8)));
  if (x_row) m_most = std::min(m_most, floor256(kSmallCap / x_row));
  mc = piece_of(l.m, m_most);
  const int64_t pieces = (l.k + Vp - 1) / Vp, slabs = (l.m + mc - 1) / mc;
  const int64_t pitch = (Vp + 7) / 8 * 8;

  Cut c;
  char *ws = nullptr, *w_at = nullptr, *x_at = nullptr, *d_at = nullptr;
  float *dx_sum = nullptr, *dw_sum = nullptr, *db_parts = nullptr, *db_sum = nullptr, *scales = nullptr;
  for (int pass = 0; pass < 2; ++pass) {
    w_at = c.take(w_row ? (l.w_trans ? Vp * w_row : l.n * pitch * d_size) : 0);
    x_at = c.take(mc * x_row);
    d_at = c.take(mc * pitch * d_size);
    dx_sum = reinterpret_cast<float*>(c.take(a.DX && pieces > 1 ? l.m * l.n * 4 : 0));
    dw_sum = reinterpret_cast<float*>(c.take(a.DW && slabs > 1 ? Vp * l.n * 4 : 0));
    db_parts = reinterpret_cast<float*>(c.take(a.DB ? (mc + 31) / 32 * Vp * 4 : 0));
    db_sum = reinterpret_cast<float*>(c.take(a.DB && slabs > 1 ? Vp * 4 : 0));
    scales = reinterpret_cast<float*>(c.take(l.type == FXTX_F16 ? kScaleBytes : 0));
    if (pass == 0) {
      const fxtx_status_t s = alloc_pooled(reinterpret_cast<void**>(&ws), c.bytes, st);
      if (s != FXTX_OK) return s;
      c.base = ws;
      c.bytes = 0;
    }
  }
  fxtx_status_t s = FXTX_OK;
  if (scales) s = status_of(launch_scales(a, l.m, l.k, scales, st));
  for (int64_t v = 0; v < l.k && s == FXTX_OK; v += Vp) {
    const int64_t n = std::min(Vp, l.k - v);
    const Part w = classes_of(l, v, n, w_at);
    for (int64_t r = 0; r < l.m && s == FXTX_OK; r += mc) {
      const int64_t rows = std::min(mc, l.m - r);
      const Part x = part_of(l.type, l.X, l.ldx, r, rows, 0, l.n, x_at);
      PackArgs packs[2];
      int count = 0;
      if (x.packed && (slabs > 1 || v == 0)) packs[count++] = x.pack;
      if (w.packed && r == 0) packs[count++] = w.pack;
      if (count) s = status_of(launch_prepare(l.type, nullptr, packs, count, dev.sm_count, st));
      // D
      PlanesProduct q;
      q.M = rows;
      q.N = n;
      q.K = l.n;
      q.A = as(x, false);
      q.B = as(w, !l.w_trans);
      q.e.bias = bias_at(l, v);
      ModeArgs<2> d;
      d.labels = labels_at(a, r);
      d.labels64 = a.labels64;
      d.count = l.k;
      d.col0 = v;
      d.lse = a.lse_in + r;
      d.g = a.g ? a.g + r : nullptr;
      d.gain = a.gain;
      d.scales = scales;
      d.D = d_at;
      d.ldd = pitch;
      d.d_planes = f32 ? rows * pitch : 0;
      d.sums = db_parts;
      d.sums_ld = n;
      if (s == FXTX_OK) s = run_slope(l.type, q, d, dev, st);
      if (s == FXTX_OK && a.DB) {
        const float* in = r > 0 ? db_sum : nullptr;
        float* keep = r + mc < l.m ? db_sum : nullptr;
        const dim3 grid((unsigned)((n + 31) / 32));
        char* db = static_cast<char*>(a.DB) + v * size;
        const int64_t parts = (rows + 31) / 32;
        switch (l.type) {
          case FXTX_F32:
            s = status_of(launch_kernel(db_join_kernel<float>, grid, 256, 0, st, db_parts, parts, n, in, keep, scales, reinterpret_cast<float*>(db)));
            break;
          case FXTX_BF16:
            s = status_of(launch_kernel(db_join_kernel<__nv_bfloat16>, grid, 256, 0, st, db_parts, parts, n, in, keep, scales,
                                        reinterpret_cast<__nv_bfloat16*>(db)));
            break;
          default:
            s = status_of(launch_kernel(db_join_kernel<__half>, grid, 256, 0, st, db_parts, parts, n, in, keep, scales, reinterpret_cast<__half*>(db)));
            break;
        }
      }
      Planes dp;
      dp.p = d_at;
      dp.rows = rows;
      dp.cols = n;
      dp.pitch = pitch;
      dp.planes = f32 ? 3 : 1;
      dp.plane_stride = rows * pitch;
      if (s == FXTX_OK && a.DX) {
        PlanesProduct t;
        t.M = rows;
        t.N = l.n;
        t.K = n;
        t.A = dp;
        t.B = as(w, l.w_trans);
        t.e.out = static_cast<char*>(a.DX) + r * a.lddx * size;
        t.e.ldo = a.lddx;
        ModeArgs<3> m;
        m.in = v > 0 ? dx_sum + r * l.n : nullptr;
        m.keep = v + Vp < l.k ? dx_sum + r * l.n : nullptr;
        m.scales = scales;
        s = run_sum(l.type, t, m, dev, st);
      }
      if (s == FXTX_OK && a.DW) {
        Planes dm = dp, xm = as(x, true);
        dm.mn_major = true;
        PlanesProduct t;
        t.M = l.w_trans ? n : l.n;
        t.N = l.w_trans ? l.n : n;
        t.K = rows;
        t.A = l.w_trans ? dm : xm;
        t.B = l.w_trans ? xm : dm;
        t.e.out = static_cast<char*>(a.DW) + (l.w_trans ? v * a.lddw : v) * size;
        t.e.ldo = a.lddw;
        ModeArgs<3> m;
        m.in = r > 0 ? dw_sum : nullptr;
        m.keep = r + mc < l.m ? dw_sum : nullptr;
        m.scales = scales;
        s = run_sum(l.type, t, m, dev, st);
      }
    }
  }
  cudaFreeAsync(ws, st);
  return s;
}

}  // namespace fxtx
