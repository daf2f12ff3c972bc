// loss_raw.cu — products of 16-bit types whose sums are kept in fp32, as they are: few rows' logits, and the gradient at few rows.
#include "product_split.cuh"
#include "product_tc.cuh"

namespace fxtx {
namespace {

TcPlan plan_of(const PlanesProduct& p, const DeviceInfo& dev) {
  return plan_product(p.M, p.N, p.K, 1, p.A.mn_major, p.B.mn_major, dev.sm_count);
}

template <typename T>
fxtx_status_t run_t(const PlanesProduct& p, float* out, const DeviceInfo& dev, cudaStream_t st) {
  const TcPlan plan = plan_of(p, dev);
  TcArgs a;
  CUtensorMap am, bm;
  const fxtx_status_t s = prepare_product<T>(p, plan, a, am, bm, LOGIT_FOLD);
  if (s != FXTX_OK) return s;
  a.part = out;
  const cudaError_t e = plan.cluster ? launch_cluster<T, true>(plan, am, bm, a, st)
                                     : launch_persistent<T, 4>(plan, am, bm, a, ModeArgs<4>{}, dev.sm_count, st);
  if (e == cudaSuccess) return FXTX_OK;
  cudaGetLastError();
  return FXTX_ERR_CUDA;
}

}  // namespace

int* raw_error_word() { return device_error_word(); }

int64_t raw_parts(const PlanesProduct& p, const DeviceInfo& dev) {
  const TcPlan plan = plan_of(p, dev);
  if (plan.cluster) return 1;
  const int64_t kb = (p.K + 127) / 128, per = (kb + plan.splits - 1) / plan.splits;
  return (kb + per - 1) / per;
}

fxtx_status_t run_raw(fxtx_type_t type, const PlanesProduct& p, float* out, const DeviceInfo& dev, cudaStream_t st) {
  if (type == FXTX_BF16) return run_t<__nv_bfloat16>(p, out, dev, st);
  return type == FXTX_F16 ? run_t<__half>(p, out, dev, st) : FXTX_ERR_UNSUPPORTED;
}

}  // namespace fxtx
