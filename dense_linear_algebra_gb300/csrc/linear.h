// linear.h — argument blocks and launchers of the fused linear layer and its gradient.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "layers.h"

namespace fxtx {

// A matrix operand of a product over an index kk: entry (i, kk) at p[i * ld + kk], or with
// mn_major at p[kk * ld + i]. plane_stride > 0: not float32 entries but their three bfloat16
// planes, plane_stride elements apart, 16-byte aligned.
struct Operand {
  const void* p = nullptr;
  int64_t ld = 0;
  bool mn_major = false;
  int64_t plane_stride = 0;
};

// What is done with a product's entry (i, j) before it is stored: out = act(acc + bias_j) + R_ij,
// acc + bias_j itself going to Z.
struct Epilogue {
  const void* bias = nullptr;
  const void* R = nullptr;
  int64_t ldr = 0;
  void* Z = nullptr;
  int64_t ldz = 0;
  void* out = nullptr;
  int64_t ldo = 0;
  int act = FXTX_ACT_NONE;
};

// A 16-bit operand as the tensor copies read it: `planes` matrices of rows x cols in memory,
// `pitch` elements from row to row and `plane_stride` from plane to plane, 16-byte aligned.
// mn_major: the rows run over kk (entry (i, kk) at row kk, column i), else over i.
struct Planes {
  const void* p = nullptr;
  int64_t rows = 0, cols = 0, pitch = 0, plane_stride = 0;
  int planes = 1;
  bool mn_major = false;
};

// The same product from planes: one of bfloat16 or float16, three bfloat16 ones of a float32 operand.
struct PlanesProduct {
  int64_t M = 0, N = 0, K = 0;
  Planes A, B;
  Epilogue e;
};
template <typename T>
fxtx_status_t run_planes(const PlanesProduct& p, const DeviceInfo& dev, cudaStream_t st);
int* product_error_word();

// How a product is laid over the tensor cores.
struct TcPlan {
  bool swap = false;  // tiles of 128 columns x bn rows of the result instead of 128 cg rows x bn columns
  bool cluster = false;  // one tile a cluster of `splits` CTAs (a power of two up to 8), each taking a part of kk
  int cg = 1, bn = 128, splits = 1;
};
TcPlan plan_product(int64_t M, int64_t N, int64_t K, int planes, bool a_mn, bool b_mn, int sm_count);
// The same among the persistent kernel's layouts, with at most `splits` parts of kk.
TcPlan plan_persistent(int64_t M, int64_t N, int64_t K, int planes, bool a_mn, bool b_mn, int sm_count, int64_t splits);

// Whether the tensor copies can read a 16-bit operand where it lies.
bool copyable(const Operand& o);
// The operand's planes (rows x cols in memory), where they will lie in `at` if it has to be packed (`bytes` of it).
Planes planes_of(const Operand& o, fxtx_type_t type, int64_t mn, int64_t k, char* at, size_t* bytes);

// A copy of a matrix with an aligned pitch: 16-bit as it is, float32 as three bfloat16 planes.
struct PackArgs {
  const void* src = nullptr;
  int64_t rows = 0, cols = 0, ld = 0;
  void* dst = nullptr;
  int64_t pitch = 0, plane_stride = 0;
};

// A layer's arguments, and its gradient's.
struct LayerArgs {
  fxtx_type_t type = FXTX_F32;
  int64_t m = 0, n = 0, k = 0;
  const void* X = nullptr;
  int64_t ldx = 0;
  const void* W = nullptr;
  int64_t ldw = 0;
  bool w_trans = false;
  Epilogue e;
};
struct GradArgs {
  const void* G = nullptr;
  int64_t ldg = 0;
  const void* Z = nullptr;
  int64_t ldz = 0;
  int act = FXTX_ACT_NONE;
  void* DX = nullptr;
  int64_t lddx = 0;
  void* DW = nullptr;
  int64_t lddw = 0;
  void* DB = nullptr;
};

// The layer and its gradient as products on the tensor cores. Allocate their own workspace.
fxtx_status_t run_linear(const LayerArgs& l, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_grad(const LayerArgs& l, const GradArgs& g, const DeviceInfo& dev, cudaStream_t st);

// Layers of 1 to kThin features and outputs, on the CUDA cores.
constexpr int kThin = 64;
bool thin_shape(int64_t n, int64_t k);
fxtx_status_t run_thin_linear(const LayerArgs& l, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_thin_grad(const LayerArgs& l, const GradArgs& g, const DeviceInfo& dev, cudaStream_t st);

// Whether a result of m rows is formed that way.
bool few_rows(fxtx_type_t type, int64_t m, bool by_column);
// float32 results of few rows on the CUDA cores: out = e(X W), W's entry (j, c) at W[j * ld + c] or by_column at
// W[c * ld + j]; X as it is, or (x_planes > 0) as its three bfloat16 planes.
constexpr int kFewByRow = 16, kFewByColumn = 8;  // rows at most
fxtx_status_t run_few(int64_t m, int64_t n, int64_t k, const void* X, int64_t ldx, int64_t x_planes, const float* W,
                      int64_t ld, bool by_column, const Epilogue& e, const DeviceInfo& dev, cudaStream_t st);

// D = G * act'(Z) and its column sums. D is written with row pitch ldd unless it is NULL (of
// float32 as three bfloat16 planes, d_planes elements apart); db unless it is NULL.
struct SlopeArgs {
  int64_t m = 0, k = 0;
  const void* G = nullptr;
  int64_t ldg = 0;
  const void* Z = nullptr;
  int64_t ldz = 0;
  int act = FXTX_ACT_NONE;
  void* D = nullptr;
  int64_t ldd = 0, d_planes = 0;
  void* db = nullptr;
  float* ws = nullptr;  // slope_ws_bytes
};
size_t slope_ws_bytes(int64_t m, int64_t k, int sm_count);
// One launch for a slope (or NULL) and up to two copies; a second one adds db's parts of many rows.
cudaError_t launch_prepare(fxtx_type_t type, const SlopeArgs* slope, const PackArgs* packs, int count, int sm_count,
                           cudaStream_t st);

}  // namespace fxtx
