// loss_stats.cu — softmax statistics of a product's rows (mode 1 of product_tc.cuh).
#include "product_tc.cuh"

namespace fxtx {

int* stats_error_word() { return device_error_word(); }

fxtx_status_t run_stats(fxtx_type_t type, const PlanesProduct& p, const ModeArgs<1>& x, const DeviceInfo& dev, cudaStream_t st) {
  switch (type) {
    case FXTX_F32: return run_mode<float, 1>(p, x, dev, st);
    case FXTX_BF16: return run_mode<__nv_bfloat16, 1>(p, x, dev, st);
    default: return run_mode<__half, 1>(p, x, dev, st);
  }
}

int64_t stat_parts(fxtx_type_t type, const PlanesProduct& p, const DeviceInfo& dev) {
  const int planes = type == FXTX_F32 ? 3 : 1;
  const TcPlan plan = plan_persistent(p.M, p.N, p.K, planes, p.A.mn_major, p.B.mn_major, dev.sm_count, 1);
  int cols = 0;  // that a thread takes
  if (planes == 3) cols = plan.bn == 64 ? TileCfg<1, 64, 3>::COLS : plan.cg == 2 ? TileCfg<2, 128, 3>::COLS : TileCfg<1, 128, 3>::COLS;
  else cols = plan.bn == 64 ? TileCfg<1, 64, 1>::COLS : plan.bn == 256 ? TileCfg<2, 256, 1>::COLS
              : plan.cg == 2 ? TileCfg<2, 128, 1>::COLS : TileCfg<1, 128, 1>::COLS;
  return (p.N + plan.bn - 1) / plan.bn * (plan.bn / cols);
}

}  // namespace fxtx
