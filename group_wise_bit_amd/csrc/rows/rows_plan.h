// Launchers of the row-wise products, one instantiation per bit width
// (rows_inst.hip).
#pragma once

#include "rows.h"

namespace qlin {

// The work-group form of a product over rows: 32 rows x 32 columns with K over
// the waves, or 64 rows x 128 columns (kSwiglu: half as many of each matrix).
struct RowsCfg {
  int height;          // rows of X per work-group
  int tiles;           // row tiles of the grid (those past the plan's end exit)
};

// Work-group columns of a product with n outputs per row.
inline int rows_cols(int n, int mode, RowsCfg c) {
  const int tiles = (n + kTile - 1) / kTile;
  if (c.height == 32) return 2 * tiles;
  return mode == kSwiglu ? tiles : (tiles + 1) / 2;
}

// Whether the grid of such a product can be launched (HIP counts threads in
// 32 bits).
inline bool rows_fits(int n, int mode, RowsCfg c) {
  return (int64_t)rows_cols(n, mode, c) * c.tiles * 512 < ((int64_t)1 << 32);
}

template <int B>
void launch_rows(const RowsArgs& a, int mode, RowsCfg c, hipStream_t st);

}  // namespace qlin
