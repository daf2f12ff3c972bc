// linear.h — argument blocks and launchers of the fused linear layer and its gradient.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "layers.h"

namespace fxtx {

// A matrix operand of a product over an index kk: entry (i, kk) at p[i * ld + kk], or with
// mn_major at p[kk * ld + i].
struct Operand {
  const void* p = nullptr;
  int64_t ld = 0;
  bool mn_major = false;
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

// C (M x N) = sum over kk < K of A(i, kk) B(j, kk), then the epilogue. Allocates its own workspace.
struct Product {
  fxtx_type_t type = FXTX_F32;
  int64_t M = 0, N = 0, K = 0;
  Operand A, B;
  Epilogue e;
};
fxtx_status_t run_product(const Product& p, const DeviceInfo& dev, cudaStream_t st);

// D = G * act'(Z) and its column sums. D is written with row pitch ldd unless it is NULL; db unless it is NULL.
struct SlopeArgs {
  fxtx_type_t type = FXTX_F32;
  int64_t m = 0, k = 0;
  const void* G = nullptr;
  int64_t ldg = 0;
  const void* Z = nullptr;
  int64_t ldz = 0;
  int act = FXTX_ACT_NONE;
  void* D = nullptr;
  int64_t ldd = 0;
  void* db = nullptr;
  float* ws = nullptr;  // slope_ws_bytes
};
size_t slope_ws_bytes(int64_t m, int64_t k, int sm_count);
cudaError_t launch_slope(const SlopeArgs& a, int sm_count, cudaStream_t st);

}  // namespace fxtx
