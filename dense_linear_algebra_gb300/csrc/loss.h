// loss.h — argument blocks of softmax cross entropy on a linear layer, and of the products that it takes.
#pragma once

#include "linear.h"

namespace fxtx {

// A row's label, -1 where it lies outside 0 .. count - 1 (the row is then left out).
__device__ __forceinline__ int64_t label_at(const void* labels, bool wide, int64_t i, int64_t count) {
  const int64_t v = wide ? static_cast<const int64_t*>(labels)[i] : (int64_t)static_cast<const int32_t*>(labels)[i];
  return v < 0 || v >= count ? -1 : v;
}

// What a product does with its sums besides the layer's epilogue (MODE 0), by mode.
template <int MODE>
struct ModeArgs {};

// Softmax statistics over the product's columns, which are col0 and on of the classes.
template <>
struct ModeArgs<1> {
  const void* labels = nullptr;
  bool labels64 = true;
  int64_t count = 0, col0 = 0;
  float2* stats = nullptr;  // [columns' part][row]: the largest z, the sum of exp(z - that)
  float* target = nullptr;  // [row] z of the label
};

// D = up g_i gain (exp(z - lse_i) - [j = label_i]), zero where the row has no label.
template <>
struct ModeArgs<2> {
  const void* labels = nullptr;
  bool labels64 = true;
  int64_t count = 0, col0 = 0;
  const float *lse = nullptr, *g = nullptr;
  float gain = 1.f;
  const float* scales = nullptr;  // up and its inverse, on the device (NULL: 1)
  void* D = nullptr;              // of the layer's type; of float32 three bfloat16 planes
  int64_t ldd = 0, d_planes = 0;
  float* sums = nullptr;          // [32 rows][column] column sums of D, unless NULL
  int64_t sums_ld = 0;
};

// out = down (C + in); or, with `keep`, keep = C + in. in, keep: fp32, as wide as the result.
template <>
struct ModeArgs<3> {
  const float* in = nullptr;
  float* keep = nullptr;
  const float* scales = nullptr;  // up and down (NULL: 1)
};

// The product with that mode, without splitting its sums but for mode 3. Rows and columns as in run_planes.
// Mode 1 writes `stat_parts` parts of the columns.
fxtx_status_t run_stats(fxtx_type_t type, const PlanesProduct& p, const ModeArgs<1>& x, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_slope(fxtx_type_t type, const PlanesProduct& p, const ModeArgs<2>& x, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_sum(fxtx_type_t type, const PlanesProduct& p, const ModeArgs<3>& x, const DeviceInfo& dev, cudaStream_t st);
int64_t stat_parts(fxtx_type_t type, const PlanesProduct& p, const DeviceInfo& dev);
// C in fp32, of 16-bit types: `raw_parts` parts of it, [part][row][column].
fxtx_status_t run_raw(fxtx_type_t type, const PlanesProduct& p, float* out, const DeviceInfo& dev, cudaStream_t st);
int64_t raw_parts(const PlanesProduct& p, const DeviceInfo& dev);
// out = mode 3's result from such parts.
fxtx_status_t join_sums(fxtx_type_t type, const ModeArgs<3>& x, void* out, int64_t ldo, int64_t rows, int64_t cols, int64_t parts,
                        const float* part, const DeviceInfo& dev, cudaStream_t st);
int* raw_error_word();
int* stats_error_word();
int* slope_error_word();
int* sum_error_word();

// The loss and its gradient.
struct LossArgs {
  const void* labels = nullptr;
  bool labels64 = true;
  float *loss = nullptr, *lse = nullptr;  // forward
  const float *lse_in = nullptr, *g = nullptr;
  float gain = 1.f;
  void* DX = nullptr;
  int64_t lddx = 0;
  void* DW = nullptr;
  int64_t lddw = 0;
  void* DB = nullptr;
};
fxtx_status_t run_loss(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_loss_grad(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_thin_loss(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_thin_loss_grad(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st);

// Many float32 rows of few classes and features, on the CUDA cores.
bool tall_loss_shape(const LayerArgs& l, bool grad);
fxtx_status_t run_tall_loss(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st);
fxtx_status_t run_tall_loss_grad(const LayerArgs& l, const LossArgs& a, const DeviceInfo& dev, cudaStream_t st);

// scales[0] = a power of two that brings |gain| max |g| over the rows with a label to 2^14 .. 2^15, scales[1] its inverse (1 and 1 where
// that is zero or not finite). What a row that is left out has for g does not count. `scales` has kScaleBytes.
constexpr int kScaleParts = 128;
constexpr int64_t kScaleBytes = (2 + kScaleParts) * 4;
cudaError_t launch_scales(const LossArgs& a, int64_t m, int64_t k, float* scales, cudaStream_t st);

}  // namespace fxtx
