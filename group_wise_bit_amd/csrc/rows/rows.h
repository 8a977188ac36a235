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
  int cols;                       // work-group columns of a row tile
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
  const float* t;                 // [splits][m][rp]: scale * A x, partial sums over K
  const uint16_t* b;              // [slots][n][rank]
  int slots, rank, rp, tsplits;   // rp: rank rounded up to 16, t is 0 from rank on
};

// A work-group's rows: positions p0 .. p0 + rows - 1 of expert e, and its column.
struct RowTile { int e, p0, rows, col; };

// Work-groups go to the 8 XCDs (each with its own L2) round-robin by their id:
// of `total` positions, numbered row tile by row tile, every XCD gets one
// contiguous range, so that the rows of a tile, and the weights of an expert,
// are fetched into one L2.
__device__ __forceinline__ int xcd_position(int total) {
  const int f = blockIdx.x, per = total / kXcds, rem = total % kXcds;
  const int xcd = f % kXcds, local = f / kXcds;
  return xcd < rem ? xcd * (per + 1) + local : rem * (per + 1) + (xcd - rem) * per + local;
}

template <int MODE>
__device__ __forceinline__ RowTile row_tile(const RowsArgs& a, int height) {
  RowTile r;
  r.e = r.p0 = r.rows = r.col = 0;
  const int tiles = MODE == kLora ? (a.m + height - 1) / height : *a.plan.ntiles;
  const int total = tiles * a.cols;
  if ((int)blockIdx.x >= total) return r;
  const int f = xcd_position(total), y = f / a.cols;
  r.col = f % a.cols;
  if constexpr (MODE == kLora) {
    r.p0 = y * height;
    r.rows = min(height, a.m - r.p0);
  } else {
    r.e = a.plan.tiles[2 * y];
    r.p0 = a.plan.tiles[2 * y + 1];
    r.rows = min(height, a.plan.offs[r.e + 1] - r.p0);
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

// The power of two 2^e that brings a row of A x into fp16's range with room for
// 22 bits in two halves: |t 2^-e| < 2^15 for the row's largest |t| (1 for a
// row of zeros or one that is not finite).
__device__ __forceinline__ float half_scale(float largest) {
  if (!(largest > 0.f) || largest > 3.402823466e38f) return 1.f;
  const int e = (int)(__builtin_bit_cast(uint32_t, largest) >> 23) - 127;   // floor(log2)
  return __builtin_bit_cast(float, (uint32_t)(max(-126, e - 14) + 127) << 23);
}

// 8 entries of one row of A x from the partial sums, in split order.
__device__ __forceinline__ void load_t8(const RowsArgs& a, const float* p, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  for (int s = 0; s < a.tsplits; ++s) {
    const f32x4 x = reinterpret_cast<const f32x4*>(p)[0], y = reinterpret_cast<const f32x4*>(p)[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[i] += x[i];
      v[4 + i] += y[i];
    }
    p += (int64_t)a.m * a.rp;
  }
}

// Adds the adapters of 32 rows to CB blocks of 32 x 32 sums (MFMA layout: lane
// (c, h), register r: row 8 (r / 4) + 4h + r % 4, column c).  row: the lane's
// row c in X, or -1; col[cb]: its column of block cb.  Each adapter that stands
// among the rows is multiplied once for all of them and added to its own rows
// alone; `part` of `parts` callers takes every parts-th adapter.  A x (fp32)
// becomes 2^e (high + low fp16 half), both halves exact products with B.
template <int CB>
__device__ __forceinline__ void add_adapters(const RowsArgs& a, int64_t row, const int (&col)[CB],
                                             int part, int parts, f32x16 (&acc)[CB]) {
  const int h = lane_id() >> 5;
  const int id = row >= 0 ? a.ids[row] : -1;
  const bool has = (uint32_t)id < (uint32_t)a.slots;
  uint32_t left = (uint32_t)__builtin_amdgcn_ballot_w64(has);
  if (left == 0) return;
  // the rows' powers of two (a lane holds half of its row's entries)
  const float* tp = a.t + (has ? row : 0) * a.rp + 8 * h;
  float top = 0.f;
  for (int q = 0; q < a.rp; q += 16) {
    float v[8];
    load_t8(a, tp + q, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) top = __builtin_fmaxf(top, __builtin_fabsf(v[i]));
  }
  const float ts = half_scale(__builtin_fmaxf(top, __shfl_xor(top, 32)));
  const float inv = 1.f / ts;              // a power of two: exact
  for (int i = 0; left != 0; ++i) {
    const int slot = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
    const uint32_t mine = (uint32_t)__builtin_amdgcn_ballot_w64(has && id == slot);
    left &= ~mine;
    if (i % parts != part) continue;
    f32x16 hi[CB], lo[CB];
    const uint16_t* bp[CB];
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
#pragma unroll
      for (int r = 0; r < 16; ++r) hi[cb][r] = lo[cb][r] = 0.f;
      bp[cb] = a.b + ((int64_t)slot * a.n + min(col[cb], a.n - 1)) * a.rank + 8 * h;
    }
    for (int q = 0; q < a.rp; q += 16) {
      float v[8];
      load_t8(a, tp + q, v);
      f16x8 th, tl;
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float x = v[e] * inv;
        th[e] = (f16)x;
        tl[e] = (f16)(x - (float)th[e]);
      }
#pragma unroll
      for (int cb = 0; cb < CB; ++cb) {
        // (past the rank A x is 0, the factor too)
        const f16x8 bf = u4_to_f16x8(q + 8 * h < a.rank ? *reinterpret_cast<const uint4*>(bp[cb] + q)
                                                        : make_uint4(0, 0, 0, 0));
        hi[cb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(th, bf, hi[cb], 0, 0, 0);
        lo[cb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(tl, bf, lo[cb], 0, 0, 0);
      }
    }
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int rr = 8 * (r >> 2) + 4 * h + (r & 3);
      const float f = __shfl(ts, rr);
      // (a select, not a product with 0: another row's infinity stays its own)
#pragma unroll
      for (int cb = 0; cb < CB; ++cb)
        acc[cb][r] += (mine >> rr) & 1 ? f * (hi[cb][r] + lo[cb][r]) : 0.f;
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
  const RowTile rt = row_tile<MODE>(a, 32);
  if (rt.rows <= 0) return;
  const int gx = rt.col;
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
  if constexpr (MODE == kLora) {
    const int cols[1] = {col};
    add_adapters<1>(a, c < rt.rows ? xr : -1, cols, wave, WAVES, acc);
  }
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

// Keeps the compiler from moving the computation of v past this point.
__device__ __forceinline__ void here(f16x8& v) { asm volatile("" : "+v"(v)); }

// -------------------------------------------------- many rows per expert --
// Work-group: 32 RB rows of one expert x 128 columns (two 64-row weight tiles;
// kSwiglu: tile t of gate and of up), 4 waves of 32 RB rows x 32 columns
// (kSwiglu: 16 columns of gate in lanes c < 16, the same 16 of up in the
// others).  A wave decodes its columns' block once, straight into MFMA B
// registers -- integers q - z, exact, no scale rounded into them -- and
// multiplies it by all RB blocks of X, read from LDS (16-byte chunks permuted
// within their row by xswz, so that operand reads fall on distinct banks).  The four MFMAs of a block start from 0 and the group's scale takes
// their sum to the fp32 accumulators, 16 fma per lane beside the next four
// MFMAs.  Two X buffers: while block j is multiplied, block j + 1's rows are
// on their way to registers and then to the other buffer; codes run two blocks
// ahead.  One barrier per block.
template <int BITS, int MODE, int RB, int D>
__global__ __launch_bounds__(256, 2) void k_rows_tiled(const RowsArgs a) {
  constexpr int WPB = 2 * BITS;
  constexpr int HW = BITS;
  constexpr int BM = 32 * RB;
  __shared__ f16x8 xs[2][BM * 8];
  const RowTile rt = row_tile<MODE>(a, BM);
  if (rt.rows <= 0) return;
  const int gx = rt.col;
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  const int c = lane & 31, h = lane >> 5;
  const uint32_t magic = vreg_const(kMagic);
  // the lane's weight row: row drow of tile dt of matrix di (a tile past the
  // matrix re-reads its last one, never stored)
  const int tiles = (a.n + kTile - 1) / kTile;
  const int tile = MODE == kSwiglu ? gx : 2 * gx + (wave >> 1);
  const int drow = MODE == kSwiglu ? 16 * wave + (c & 15) : 32 * (wave & 1) + c;
  const int di = MODE == kSwiglu ? c >> 4 : 0;
  const int dt = min(tile, tiles - 1);
  const uint32_t* wsrc = (di ? a.codes[1] : a.codes[0]) + rt.e * a.code_step +
                         ((int64_t)dt * a.kb * kTile + drow) * WPB;
  const int64_t mt = rt.e * a.meta_step + (int64_t)dt * a.G * kTile + drow;
  const uint16_t* ssrc = (di ? a.scale[1] : a.scale[0]) + mt;
  const uint8_t* zsrc = (di ? a.zero[1] : a.zero[0]) + mt;
  const int t8 = tid >> 3, xk = tid & 7;
  const uint16_t* xsrc[RB];
#pragma unroll
  for (int i = 0; i < RB; ++i) {
    const int r = t8 + 32 * i;
    xsrc[i] = a.X + x_row<MODE>(a, rt.p0 + (r < rt.rows ? r : 0)) * a.ldx + 8 * xk;
  }
  const int xw = 8 * t8 + xswz(t8, xk);      // (rows 32 apart: the same place in their row)

  uint32_t wl[D][HW];
  uint16_t sr[D];
  int zc[D];
  f16x8 xg[D][RB];
  auto request_x = [&](auto S, int j) __attribute__((always_inline)) {
    constexpr int u = decltype(S)::value;
    const int jj = min(j, a.kb - 1);
#pragma unroll
    for (int i = 0; i < RB; ++i)
      xg[u][i] = *reinterpret_cast<const f16x8*>(xsrc[i] + (int64_t)jj * kBlock);
  };
  auto request_w = [&](auto S, int j) __attribute__((always_inline)) {
    constexpr int u = decltype(S)::value;
    const int jj = min(j, a.kb - 1);
    load_half<BITS>(wsrc + (int64_t)jj * kTile * WPB, h, wl[u]);
    const int64_t g = (a.G == 1) ? 0 : jj;
    sr[u] = ssrc[g * kTile];
    zc[u] = zsrc[g * kTile];
  };
  auto store_x = [&](auto S, int b) __attribute__((always_inline)) {
    constexpr int u = decltype(S)::value;
#pragma unroll
    for (int i = 0; i < RB; ++i) xs[b][xw + 256 * i] = xg[u][i];
  };
  f32x16 acc[RB];
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[rb][r] = 0.f;
  f16x8 bv[2][4];
  float scl[2];
  f32x16 blk[2];               // sums of one block and 32 rows, not yet scaled
#pragma unroll
  for (int r = 0; r < 16; ++r) blk[0][r] = blk[1][r] = 0.f;
  scl[1] = 0.f;
  static_for<0, D>([&](auto S) __attribute__((always_inline)) {
    request_w(S, decltype(S)::value);
    request_x(S, decltype(S)::value);
  });
  const std::integral_constant<int, 0> S0;
  {
    const DeqT<BITS> d = make_deq_b<BITS>(1.f, zc[0]);
#pragma unroll
    for (int q = 0; q < 4; ++q) bv[0][q] = int_half<BITS>(wl[0], q, d, magic);
    scl[0] = h2f(sr[0]);
    store_x(S0, 0);
    request_w(S0, D);
  }
  lds_barrier();
  // block j (slot U of D): from X buffer and operand registers j % 2; block
  // j + 1's codes and rows wait in slot U + 1, slot U's rows are free
  auto step = [&](auto U, int j) __attribute__((always_inline)) {
    constexpr int u = decltype(U)::value, b = u & 1;
    const std::integral_constant<int, (u + 1) % D> N;
    constexpr int n = (u + 1) % D;
    f16x8 av[2][4];
    auto read_a = [&](int rb) __attribute__((always_inline)) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        av[rb & 1][q] = xs[b][8 * (32 * rb + c) + xswz(c, 4 * h + q)];
    };
    auto scale_block = [&](int rb, float s) __attribute__((always_inline)) {
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[rb][r] = __builtin_fmaf(s, blk[rb & 1][r], acc[rb][r]);
    };
    read_a(0);
    request_x(U, j + D);
    const DeqT<BITS> d = make_deq_b<BITS>(1.f, zc[n]);
    // the previous block's last rows, while this block's first operands arrive
    scale_block(RB - 1, scl[1 - b]);
    scl[1 - b] = h2f(sr[n]);
    asm volatile("" : "+v"(scl[1 - b]));
#pragma unroll
    for (int rb = 0; rb < RB; ++rb) {
      if (rb + 1 < RB) read_a(rb + 1);
      __builtin_amdgcn_sched_barrier(0);
      const f32x16 none = {};
#pragma unroll
      for (int q = 0; q < 4; ++q)
        blk[rb & 1] = __builtin_amdgcn_mfma_f32_32x32x16_f16(
            av[rb & 1][q], bv[b][q], q == 0 ? none : blk[rb & 1], 0, 0, 0);
#pragma unroll
      for (int q = rb * 4 / RB; q < (rb + 1) * 4 / RB; ++q) {
        bv[1 - b][q] = int_half<BITS>(wl[n], q, d, magic);
        here(bv[1 - b][q]);
      }
      if (rb > 0) scale_block(rb - 1, scl[b]);
      __builtin_amdgcn_sched_barrier(0);
    }
    store_x(N, 1 - b);
    request_w(N, j + 1 + D);
    lds_barrier();
  };
  int j0 = 0;
  for (; j0 + D <= a.kb; j0 += D)
    static_for<0, D>([&](auto U) __attribute__((always_inline)) {
      step(U, j0 + decltype(U)::value);
    });
  static_for<0, D - 1>([&](auto U) __attribute__((always_inline)) {
    if (j0 + decltype(U)::value < a.kb) step(U, j0 + decltype(U)::value);
  });
  {
    const float s = a.kb & 1 ? scl[0] : scl[1];
#pragma unroll
    for (int r = 0; r < 16; ++r)
      acc[RB - 1][r] = __builtin_fmaf(s, blk[(RB - 1) & 1][r], acc[RB - 1][r]);
  }

  const int col = tile * kTile + drow;
  if constexpr (MODE == kLora) {
    const int cols[1] = {col};
#pragma unroll
    for (int rb = 0; rb < RB; ++rb)
      add_adapters<1>(a, 32 * rb + c < rt.rows ? x_row<MODE>(a, rt.p0 + 32 * rb + c) : -1, cols, 0,
                      1, reinterpret_cast<f32x16(&)[1]>(acc[rb]));
  }
#pragma unroll
  for (int rb = 0; rb < RB; ++rb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      const int row = 32 * rb + 8 * (r >> 2) + 4 * h + (r & 3);
      if constexpr (MODE == kSwiglu) {
        const float u = __shfl_xor(acc[rb][r], 16);
        if (row >= rt.rows || c >= 16) continue;
        const float hv = silu(acc[rb][r]) * u;
        a.y16[(int64_t)(rt.p0 + row) * a.ldy + col] = __builtin_bit_cast(uint16_t, (f16)hv);
      } else {
        if (row >= rt.rows || col >= a.n) continue;
        const int64_t out = MODE == kDown ? a.plan.order[rt.p0 + row] : x_row<MODE>(a, rt.p0 + row);
        const float v = MODE == kDown ? a.weights[out] * acc[rb][r] : acc[rb][r];
        if (MODE == kDown || a.y != nullptr) a.y[out * a.ldy + col] = v;
        if (MODE == kLora && a.y16 != nullptr)
          a.y16[out * a.ldy + col] = __builtin_bit_cast(uint16_t, (f16)v);
      }
    }
}

}  // namespace qlin
