// One bit width's row-wise products, compiled as its own object with
// -DQLIN_INST_BITS=<width>.
#include "rows_plan.h"

namespace qlin {

constexpr int kB = QLIN_INST_BITS;

template <int B>
void launch_rows(const RowsArgs& args, int mode, RowsCfg c, hipStream_t st) {
  RowsArgs a = args;
  a.cols = rows_cols(a.n);
  const dim3 grid((unsigned)((int64_t)a.cols * c.tiles));
  constexpr int W = 8;
  const dim3 block(W * 64);
  if (mode == kSwiglu) {
    hipLaunchKernelGGL((k_rows_ksplit<B, kSwiglu, W, 1>), grid, block, 0, st, a);
  } else if (mode == kDown) {
    hipLaunchKernelGGL((k_rows_ksplit<B, kDown, W, 2>), grid, block, 0, st, a);
  } else {
    hipLaunchKernelGGL((k_rows_ksplit<B, kLora, W, 2>), grid, block, 0, st, a);
  }
}

template void launch_rows<kB>(const RowsArgs&, int, RowsCfg, hipStream_t);

}  // namespace qlin
