// One bit width's row-wise products, compiled as its own object with
// -DQLIN_INST_BITS=<width>.
#include "rows_plan.h"

namespace qlin {

constexpr int kB = QLIN_INST_BITS;

template <int B, int MODE, bool DOTS>
void launch_ksplit(const RowsArgs& a, RowsCfg c, dim3 grid, hipStream_t st) {
  constexpr int U = MODE == kSwiglu && B > 4 ? 1 : 2;   // by the registers of a block
  const dim3 block(64 * c.waves);
  if (c.half) hipLaunchKernelGGL((k_rows_ksplit<B, MODE, 8, 1, 2, DOTS>), grid, block, 0, st, a);
  else if (c.waves == 8) hipLaunchKernelGGL((k_rows_ksplit<B, MODE, 8, 2, U, DOTS>), grid, block, 0, st, a);
  else hipLaunchKernelGGL((k_rows_ksplit<B, MODE, 4, 2, U, DOTS>), grid, block, 0, st, a);
}

template <int B, int MODE>
void launch_mode(const RowsArgs& a, RowsCfg c, hipStream_t st) {
  const dim3 grid((unsigned)((int64_t)a.cols * c.tiles)), block(rows_threads(c));
  if constexpr (MODE == kSwiglu || MODE == kToken) {
    if (c.height == 1) {
      if (!c.half) hipLaunchKernelGGL((k_rows_gemv<B, MODE, 4, 8, 4>), grid, block, 0, st, a);
      else if (c.waves == 16) hipLaunchKernelGGL((k_rows_gemv<B, MODE, 8, 16, 4>), grid, block, 0, st, a);
      else hipLaunchKernelGGL((k_rows_gemv<B, MODE, 8, 8, 4>), grid, block, 0, st, a);
      return;
    }
  }
  if constexpr (MODE != kToken) {
    if (c.height == 64) {
      hipLaunchKernelGGL((k_rows_tiled<B, MODE>), grid, block, 0, st, a);
      return;
    }
    if constexpr (MODE == kLora) {
      if (c.dots) {
        launch_ksplit<B, MODE, true>(a, c, grid, st);
        return;
      }
    }
    launch_ksplit<B, MODE, false>(a, c, grid, st);
  }
}

template <int B>
void launch_rows(const RowsArgs& args, int mode, RowsCfg c, hipStream_t st) {
  RowsArgs a = args;
  a.cols = rows_cols(a.n, mode, c);
  if (mode == kSwiglu) launch_mode<B, kSwiglu>(a, c, st);
  else if (mode == kDown) launch_mode<B, kDown>(a, c, st);
  else if (mode == kLora) launch_mode<B, kLora>(a, c, st);
  else launch_mode<B, kToken>(a, c, st);
}

template void launch_rows<kB>(const RowsArgs&, int, RowsCfg, hipStream_t);

}  // namespace qlin
