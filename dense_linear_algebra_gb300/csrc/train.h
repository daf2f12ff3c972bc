// train.h — argument blocks and launchers of what training a classifier takes besides its layers: layer norm, the
// embedding lookup, softmax cross entropy on a linear layer, each with its gradient.
#pragma once

#include <cstdint>
#include <cuda_runtime.h>

#include "layers.h"

namespace fxtx {

// out = (x - mean) rstd w + b over the rows of X (w, b may be NULL: ones, zeros), and its gradient.
struct NormArgs {
  int64_t m = 0, n = 0;
  const void* X = nullptr;
  int64_t ldx = 0;
  const void *w = nullptr, *b = nullptr;
  float eps = 0.f;
  void* out = nullptr;
  int64_t ldo = 0;
  float *mean = nullptr, *rstd = nullptr;  // written by the forward pass unless NULL
  // the gradient's
  const float *mean_in = nullptr, *rstd_in = nullptr;
  const void* G = nullptr;
  int64_t ldg = 0;
  const void* R = nullptr;  // the gradient that arrives on the residual path
  int64_t ldr = 0;
  void* DX = nullptr;
  int64_t lddx = 0;
  void *DW = nullptr, *DB = nullptr;
  float* part = nullptr;  // [CTAs][2][n] column sums
};
int* norm_error_word();
fxtx_status_t run_norm(fxtx_type_t type, const NormArgs& a, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_norm_grad(fxtx_type_t type, const NormArgs& a, const DeviceInfo& dev, cudaStream_t st);

// out_i = scale E[ids_i] (zeros for an id outside 0 .. count - 1), and its gradient dE_v = scale * the sum of the
// rows of G with id v.
struct EmbedArgs {
  int64_t m = 0, n = 0, count = 0;
  const void* ids = nullptr;
  bool ids64 = true;
  float scale = 1.f;
  const void* src = nullptr;  // E, or G
  int64_t lds = 0;
  void* out = nullptr;  // the rows, or dE
  int64_t ldo = 0;
};
fxtx_status_t run_embed(fxtx_type_t type, const EmbedArgs& a, const DeviceInfo& dev, cudaStream_t st);
int* embed_error_word();
fxtx_status_t run_embed_grad(fxtx_type_t type, const EmbedArgs& a, const DeviceInfo& dev, cudaStream_t st);

}  // namespace fxtx
