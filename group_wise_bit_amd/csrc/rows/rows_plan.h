// Launchers of the row-wise products, one instantiation per bit width
// (rows_inst.hip).
#pragma once

#include "rows.h"

namespace qlin {

// The work-group form of a product over rows: one row x 8 or 16 columns (kSwiglu,
// kToken), up to 32 rows x 32 or 64 columns with K over 4 or 8 waves, or 64
// rows x 256 columns (kSwiglu: half as many of each matrix).
struct RowsCfg {
  int height;          // rows of X per work-group: 1, 32 or 64
  int tiles;           // row tiles of the grid (those past the plan's end exit)
  int waves;           // (1 and 32 rows) waves per work-group
  bool half;           // 32 columns per work-group (32 rows), 8 (one row)
  bool dots;           // (32 rows) adapters of rank <= kDotRank, rows as they come
};

// (32 rows) The form for about `groups` work-groups of 64 columns.  Few of them
// take K over 8 waves, or 32 columns each: of 64 against 32 columns 40 rows on 2048 x
// 2048 (64 work-groups) took 13.5 : 11.7 us, on 4096 x 4096 (128) 18.6 : 16.4, on 6144 x
// 4096 (192) 20.5 : 21.7, 333 rows on 896 x 4864 (154) 17 : 24, beyond a work-group
// per CU.  Of 8 against 4 waves 100 rows on 4096 x 4096 (256) took 19.8 :
// 21.4 us, on 6144 x 4096 (384) 36.1 : 34.9, on 8192 x 512 (512) 15.8 : 12.7; 27 rows
// through 8 of 128 experts of 512 x 1024 (1024) 51 : 37.
inline void ksplit_form(RowsCfg& c, int64_t groups) {
  c.half = groups <= 128;
  c.waves = groups < 320 ? 8 : 4;
}

// (1 row) The form for `items` K-blocks and `groups` work-groups of 16 columns: 8
// columns where 16 would not reach every CU, and then 16 waves for a long K.  Of 16
// against 8 columns a row through 4 of 64 experts of 256 x 512 took 7.9 : 6.9 us, 3 rows
// through 8 of 64 of 1024 x 2048 31.0 : 33.3; a row through those (first product 512
// work-groups of 16 columns, second 128, of 128 blocks) 14.2 by this rule, 16.7 with
// 16 columns and 8 waves in both, 18.7 with 16 waves in both; of 16 against 8 waves a
// row through 2 of 8 experts of 512 x 1024 8.1 : 6.9.
inline void gemv_form(RowsCfg& c, int items, int64_t groups) {
  c.half = groups < 256;
  c.waves = c.half && items > 32 ? 16 : 8;
}

// Work-group columns of a product with n outputs per row.
inline int rows_cols(int n, int mode, RowsCfg c) {
  const int tiles = (n + kTile - 1) / kTile;
  if (c.height == 1) return (c.half ? 8 : 4) * tiles;
  if (c.height == 32) return c.half ? 2 * tiles : tiles;
  return mode == kSwiglu ? (tiles + 1) / 2 : (tiles + 3) / 4;
}

inline int rows_threads(RowsCfg c) { return c.height == 64 ? 256 : 64 * c.waves; }

// Whether the grid of such a product can be launched (HIP counts threads in
// 32 bits).
inline bool rows_fits(int n, int mode, RowsCfg c) {
  return (int64_t)rows_cols(n, mode, c) * c.tiles * rows_threads(c) < ((int64_t)1 << 32);
}

// Whether the 64-row form is used for about `tiles` row tiles of m rows of
// stride ld, k values each.  It takes 0.5 us per K-block and work-group on a CU
// however few there are, so it needs a work-group for every other CU: of 32-row
// against 64-row tiles, adapters on 4096 x 4096 (4 bits) took 58 : 73 us for 512
// rows (128 work-groups), 82 : 75 us for 768; on 2048 x 2048 40 : 62 us for 512
// (64), 69 : 63 us for 1024; 8 experts of 1024 x 512 33 : 35 us at 64 rows each (48),
// 45 : 37 us at 128 (80), of 2048 x 1024 44 : 50 us at 64 (96), 67 : 53 us at 128 (160), 4
// of 2048 x 768 43 : 47 us at 128 (60).  It reads X by 32-bit offsets.
inline bool tiled_form(int n, int mode, int64_t tiles, int64_t m, int64_t ld, int64_t k) {
  RowsCfg c{};
  c.height = 64;
  return rows_cols(n, mode, c) * tiles >= 144 && ((m - 1) * ld + k) * 2 < ((int64_t)1 << 32);
}

template <int B>
void launch_rows(const RowsArgs& a, int mode, RowsCfg c, hipStream_t st);

}  // namespace qlin
