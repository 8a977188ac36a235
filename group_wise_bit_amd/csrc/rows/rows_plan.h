// Launchers of the row-wise products, one instantiation per bit width
// (rows_inst.hip).
#pragma once

#include "rows.h"

namespace qlin {

// The work-group form of a product over rows.
struct RowsCfg {
  int height;          // rows of X per work-group
  int tiles;           // row tiles of the grid (those past the plan's end exit)
};

// Work-group columns of a product with n outputs per row.
inline int rows_cols(int n) { return 2 * ((n + kTile - 1) / kTile); }

// Whether the grid of such a product can be launched (HIP counts threads in
// 32 bits).
inline bool rows_fits(int n, RowsCfg c) {
  return (int64_t)rows_cols(n) * c.tiles * 512 < ((int64_t)1 << 32);
}

template <int B>
void launch_rows(const RowsArgs& a, int mode, RowsCfg c, hipStream_t st);

}  // namespace qlin
