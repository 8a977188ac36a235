// One bit width's row-wise products, compiled as its own object with
// -DQLIN_INST_BITS=<width>.
#include "rows_plan.h"

namespace qlin {

constexpr int kB = QLIN_INST_BITS;


template <int B, int MODE>
void launch_mode(const RowsArgs& a, RowsCfg c, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.cols * c.tiles));
  if (c.height == 32) {
    constexpr int W = 8, U = MODE == kSwiglu ? 1 : 2;
    hipLaunchKernelGGL((k_rows_ksplit<B, MODE, W, U>), grid, dim3(W * 64), 0, st, a);
  } else {
    hipLaunchKernelGGL((k_rows_tiled<B, MODE, 2, 4>), grid, dim3(256), 0, st, a);
  }
}

template <int B>
void launch_rows(const RowsArgs& args, int mode, RowsCfg c, hipStream_t st) {
  RowsArgs a = args;
  a.cols = rows_cols(a.n, mode, c);
  if (mode == kSwiglu) launch_mode<B, kSwiglu>(a, c, st);
  else if (mode == kDown) launch_mode<B, kDown>(a, c, st);
  else launch_mode<B, kLora>(a, c, st);
}

template void launch_rows<kB>(const RowsArgs&, int, RowsCfg, hipStream_t);

}  // namespace qlin
