// Kernels whose weights differ from row to row of a batch: routing to experts,
// the experts' gated MLP over packed weights, low-rank adapters beside one
// packed projection (gfx950, wave64).
#pragma once

#include "../kernels.h"

namespace qlin {

constexpr int kMaxExperts = 512;
constexpr int kMaxTopK = 32;

// Rows ordered by expert (k_rows_plan).
struct RowPlan {
  int32_t* offs;      // [buckets + 2]: first position of each bucket, then the count
  int32_t* order;     // [count]: position -> index
  int32_t* tiles;     // [2 * ntiles]: bucket, first position
  int32_t* ntiles;    // [1]
};

// -------------------------------------------------------- weight operand --
// The 8 codes of a lane's half block for instruction s as fp16 q - z: integers
// of at most 9 bits, exact.  The group's scale multiplies the block's sums.
template <int BITS>
__device__ __forceinline__ f16x8 int_half(const uint32_t* wl, int s, const DeqT<BITS>& d,
                                          uint32_t magic) {
  f16x2 o[4];
  if constexpr (BITS >= 5 && BITS <= 7) {
    f16x2 hi[4];
    qz_chunk4(wl[s], d.lo, magic, o);
    if constexpr (BITS == 5) {
      qz_chunk1(wl[4] >> (4 * s), d.hi, magic, hi);
    } else if constexpr (BITS == 6) {
      const uint32_t v = wl[4 + (s >> 1)];
      qz_chunk2((s & 1) ? (v >> 8) : v, d.hi, magic, hi);
    } else {
      const int u = s >> 1;
      const uint32_t L = wl[4 + u];
      const uint32_t Hu = u ? __builtin_amdgcn_alignbit(wl[6], wl[6], 8) : wl[6];
      qz_chunk3((s & 1) ? (L >> 8) : L, (s & 1) ? (Hu >> 1) : Hu, d.hi, magic, hi);
    }
    const f16x2 sixteen = {(f16)16.0f, (f16)16.0f};
#pragma unroll
    for (int p = 0; p < 4; ++p) o[p] = __builtin_elementwise_fma(hi[p], sixteen, o[p]);
  } else if constexpr (BITS == 4) {
    qz_chunk4(wl[s], d, magic, o);
  } else if constexpr (BITS == 2) {
    const uint32_t v = wl[s >> 1];
    qz_chunk2((s & 1) ? (v >> 8) : v, d, magic, o);
  } else if constexpr (BITS == 8) {
    qz_chunk8(wl[2 * s], wl[2 * s + 1], d, o);
  } else {
    const int u = s >> 1;
    const uint32_t L = wl[u];
    const uint32_t Hu = u ? __builtin_amdgcn_alignbit(wl[2], wl[2], 8) : wl[2];
    qz_chunk3((s & 1) ? (L >> 8) : L, (s & 1) ? (Hu >> 1) : Hu, d, magic, o);
  }
  f16x8 r;
#pragma unroll
  for (int p = 0; p < 4; ++p) {
    r[2 * p] = o[p].x;
    r[2 * p + 1] = o[p].y;
  }
  return r;
}

// ------------------------------------------------------------------ launches --
// What a product over rows does with its sums:
//   kSwiglu  two matrices (gate, up): fp16 silu(g) * u, one row per position
//   kDown    fp32 weights[index] * sum, one row per index (pair of token and slot)
//   kLora    sum + the row's adapter, fp32 and / or fp16
enum RowsMode { kSwiglu = 0, kDown = 1, kLora = 2 };

struct RowsArgs {
  const uint32_t* codes[2];
  const uint16_t* scale[2];
  const uint8_t* zero[2];
  int64_t code_step, meta_step;   // words / entries from one expert to the next
  int n, kb, G;
  int cols;                       // work-group columns: blockIdx.x = row tile * cols + column
  const uint16_t* X;
  int64_t ldx;
  int m, top_k;
  RowPlan plan;                   // order null: positions are rows themselves
  const float* weights;           // kDown
  uint16_t* y16;                  // kSwiglu: h; kLora: Y16 or null
  float* y;                       // kDown: partial rows; kLora: Y or null
  int64_t ldy;
  // kLora
  const int32_t* ids;
  const uint16_t* t;              // [m][2][rp]: the high and low halves of A x
  const float* tscale;            // [m]: their power of two
  const uint16_t* b;              // [slots][n][rank]
  int slots, rank, rp;            // rp: rank rounded up to 16
};

// A work-group's rows: positions p0 .. p0 + rows - 1 of expert e.
struct RowTile { int e, p0, rows; };

template <int MODE>
__device__ __forceinline__ RowTile row_tile(const RowsArgs& a, int y, int height) {
  RowTile r;
  if constexpr (MODE == kLora) {
    r.e = 0;
    r.p0 = y * height;
    r.rows = min(height, a.m - r.p0);
  } else {
    r.rows = 0;
    r.e = r.p0 = 0;
    if (y < *a.plan.ntiles) {
      r.e = a.plan.tiles[2 * y];
      r.p0 = a.plan.tiles[2 * y + 1];
      r.rows = min(height, a.plan.offs[r.e + 1] - r.p0);
    }
  }
  return r;
}

// The X row of a position.
template <int MODE>
__device__ __forceinline__ int64_t x_row(const RowsArgs& a, int p) {
  if constexpr (MODE == kSwiglu) return a.plan.order[p] / a.top_k;
  else if constexpr (MODE == kDown) return p;
  else return a.plan.order != nullptr ? a.plan.order[p] : p;
}

// Adds the adapters of 32 rows to a 32 x 32 block of sums (MFMA layout: lane
// (c, h), register r: row 8 (r / 4) + 4h + r % 4, column col of the lane).
// row: this lane's row c of X, or -1.  Each adapter that stands among the rows
// is multiplied once for all 32 rows and added to its own alone; `part` of
// `parts` callers takes every parts-th of them.
__device__ __forceinline__ void add_adapters(const RowsArgs& a, int64_t row, int col, int part,
                                             int parts, f32x16& acc) {
  const int lane = lane_id(), h = lane >> 5;
  const int id = row >= 0 ? a.ids[row] : -1;
  const bool has = (uint32_t)id < (uint32_t)a.slots;
  const float ts = has ? a.tscale[row] : 0.f;
  uint32_t left = (uint32_t)__builtin_amdgcn_ballot_w64(has);
  for (int i = 0; left != 0; ++i) {
    const int first = __builtin_ctz(left);
    const int slot = __builtin_amdgcn_readlane(id, first);
    const uint32_t mine = (uint32_t)__builtin_amdgcn_ballot_w64(has && id == slot);
    left &= ~mine;
    if (i % parts != part) continue;
    f32x16 hi, lo;
#pragma unroll
    for (int r = 0; r < 16; ++r) hi[r] = lo[r] = 0.f;
    const uint16_t* tp = a.t + (has ? row : 0) * 2 * a.rp + 8 * h;
    const uint16_t* bp = a.b + ((int64_t)slot * a.n + min(col, a.n - 1)) * a.rank;
    for (int q = 0; q < a.rp; q += 16) {
      // (past the rank: the halves of A x are 0, the factor too)
      uint4 bv = make_uint4(0, 0, 0, 0);
      if (q + 8 * h < a.rank) bv = *reinterpret_cast<const uint4*>(bp + q + 8 * h);
      const f16x8 bf = u4_to_f16x8(bv);
      hi = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          u4_to_f16x8(*reinterpret_cast<const uint4*>(tp + q)), bf, hi, 0, 0, 0);
      lo = __builtin_amdgcn_mfma_f32_32x32x16_f16(
          u4_to_f16x8(*reinterpret_cast<const uint4*>(tp + a.rp + q)), bf, lo, 0, 0, 0);
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int rr = 8 * (r >> 2) + 4 * h + (r & 3);
      const float f = __shfl(ts, rr);
      // (a select, not a product with 0: another row's infinity stays its own)
      acc[r] += (mine >> rr) & 1 ? f * (hi[r] + lo[r]) : 0.f;
    }
  }
}

// --------------------------------------------------- few rows per expert --
// Work-group: up to 32 rows of one expert x 32 columns (half a 64-row weight
// tile; kSwiglu: of gate and of up).  Its waves take the K-blocks w, w +
// WAVES, ..., U at a time with every load in flight before the first decode,
// and add their sums in LDS in wave order.  Bound by the weights' bytes.
// Lane (c, h) supplies X row c / weight row c and K positions 32h + 8s .. +7.
template <int BITS, int MODE, int WAVES, int U>
__global__ __launch_bounds__(WAVES * 64) void k_rows_ksplit(const RowsArgs a) {
  constexpr int WPB = 2 * BITS;
  constexpr int HW = BITS;                   // words of a half block
  constexpr int NM = MODE == kSwiglu ? 2 : 1;
  constexpr int NT = WAVES * 64;
  constexpr int PT = 1024 / NT;              // outputs per thread
  static_assert(16 % WAVES == 0, "reduction split");
  __shared__ float red[WAVES][1024];
  const int gy = blockIdx.x / a.cols, gx = blockIdx.x % a.cols;
  const RowTile rt = row_tile<MODE>(a, gy, 32);
  if (rt.rows <= 0) return;
  const int lane = lane_id(), wave = wave_id();
  const int c = lane & 31, h = lane >> 5;
  const int t = gx >> 1, cb = gx & 1;
  const uint32_t magic = vreg_const(kMagic);
  // rows past the tile read its first row (never stored)
  const int64_t xr = x_row<MODE>(a, rt.p0 + (c < rt.rows ? c : 0));
  const uint16_t* xrow = a.X + xr * a.ldx + 32 * h;
  const uint32_t* wsrc[NM];
  const uint16_t* ssrc[NM];
  const uint8_t* zsrc[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    wsrc[i] = a.codes[i] + rt.e * a.code_step + ((int64_t)t * a.kb * kTile + 32 * cb + c) * WPB;
    const int64_t mt = rt.e * a.meta_step + (int64_t)t * a.G * kTile + 32 * cb + c;
    ssrc[i] = a.scale[i] + mt;
    zsrc[i] = a.zero[i] + mt;
  }
  f32x16 acc[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[i][r] = 0.f;
  for (int jb = wave; jb < a.kb; jb += WAVES * U) {
    f16x8 xa[U][4];
    uint32_t wl[U][NM][HW];
    uint16_t sr[U][NM];
    int zc[U][NM];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(jb + WAVES * u, a.kb - 1);     // past the range: re-read, not used
      const f16x8* xp = reinterpret_cast<const f16x8*>(xrow + (int64_t)j * kBlock);
#pragma unroll
      for (int s = 0; s < 4; ++s) xa[u][s] = xp[s];
      const int64_t g = (a.G == 1) ? 0 : j;
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        load_half<BITS>(wsrc[i] + (int64_t)j * kTile * WPB, h, wl[u][i]);
        sr[u][i] = ssrc[i][g * kTile];
        zc[u][i] = zsrc[i][g * kTile];
      }
    }
    loads_issued();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (jb + WAVES * u >= a.kb) break;
#pragma unroll
      for (int i = 0; i < NM; ++i) {
        const DeqT<BITS> d = make_deq_b<BITS>(1.f, zc[u][i]);
        f32x16 blk;
#pragma unroll
        for (int r = 0; r < 16; ++r) blk[r] = 0.f;
#pragma unroll
        for (int s = 0; s < 4; ++s)
          blk = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[u][s], int_half<BITS>(wl[u][i], s, d, magic),
                                                       blk, 0, 0, 0);
        const float sc = h2f(sr[u][i]);
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][r] = __builtin_fmaf(sc, blk[r], acc[i][r]);
      }
    }
  }
  const int col = t * kTile + 32 * cb + c;
  if constexpr (MODE == kLora)
    add_adapters(a, c < rt.rows ? xr : -1, col, wave, WAVES, acc[0]);
  // thread (wave, lane) finishes registers wave, wave + WAVES, ...
  float v[NM][PT];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int r = 0; r < 16; ++r) red[wave][64 * r + lane] = acc[i][r];
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PT; ++p) {
      float sum = red[0][64 * (wave + WAVES * p) + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum += red[w][64 * (wave + WAVES * p) + lane];
      v[i][p] = sum;
    }
  }
#pragma unroll
  for (int p = 0; p < PT; ++p) {
    const int r = wave + WAVES * p;
    const int row = 8 * (r >> 2) + 4 * h + (r & 3);
    if (row >= rt.rows || col >= a.n) continue;
    if constexpr (MODE == kSwiglu) {
      const float hv = silu(v[0][p]) * v[1][p];
      a.y16[(int64_t)(rt.p0 + row) * a.ldy + col] = __builtin_bit_cast(uint16_t, (f16)hv);
    } else if constexpr (MODE == kDown) {
      const int64_t pair = a.plan.order[rt.p0 + row];
      a.y[pair * a.ldy + col] = a.weights[pair] * v[0][p];
    } else {
      const int64_t o = x_row<MODE>(a, rt.p0 + row) * a.ldy + col;
      if (a.y != nullptr) a.y[o] = v[0][p];
      if (a.y16 != nullptr) a.y16[o] = __builtin_bit_cast(uint16_t, (f16)v[0][p]);
    }
  }
}

}  // namespace qlin
