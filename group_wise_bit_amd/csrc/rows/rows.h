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
  int32_t* order;     // [count]: position -> index
  int4* tiles;        // [ntiles]: bucket, first position, rows
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

// p + a wave-uniform offset, then a lane's 32-bit offset: the form in which a
// load takes its base from scalar registers and costs no vector address.
template <typename T>
__device__ __forceinline__ const T* lane_ptr(const T* p, int64_t uniform, uint32_t lane_off) {
  return reinterpret_cast<const T*>(reinterpret_cast<const char*>(p + uniform) +
                                    lane_off * (uint32_t)sizeof(T));
}

// ------------------------------------------------------------------ launches --
// What a product over rows does with its sums:
//   kSwiglu  two matrices (gate, up): silu(g) * u as two fp16 halves, one row per
//            position (put_halves)
//   kDown    fp32 weights[index] * sum, one row per index (pair of token and slot)
//   kLora    sum + the row's adapter, fp32 and / or fp16
//   kToken   one token: its slots' sums times their weights, fp32 and / or fp16
enum RowsMode { kSwiglu = 0, kDown = 1, kLora = 2, kToken = 3 };

// h = silu(g) * u goes to the down product as a high and a low fp16 half: the low one is
// what rounding to the high one left, so that the two hold 22 bits of it (in steps of
// 2^-24 below 2^-3; infinite from 65520 on, as fp16 is).  Each half's products with q - z
// are exact.  One half left fp32 outputs off by 2.1e-4 (rms, relative), two by 2e-7; two
// cost twice the MFMAs of the down product: 374 : 440 us for 16384 pairs through 32 experts of
// 2 x 1408 x 2048, 136 : 149 for 1018 through 16 of 1792 x 4096 at 8 bits, 32.7 : 34.4 for
// 216 through 128 of 512 x 1024, 12.9 : 13.6 for a row through 8 of 1024 x 2048.
// A row holds K-block after K-block, 64 high halves and the 64 low ones behind.
constexpr int kHalvesBlock = 2 * kBlock;
__device__ __forceinline__ void put_halves(uint16_t* row, int col, float h) {
  const f16 hi = (f16)h;
  const f16 lo = (f16)(h - (float)hi);
  uint16_t* p = row + (int64_t)(col / kBlock) * kHalvesBlock + col % kBlock;
  p[0] = __builtin_bit_cast(uint16_t, hi);
  // (an infinite high half stands alone: the difference would be NaN or infinite again)
  p[kBlock] = __builtin_isinf((float)hi) ? 0 : __builtin_bit_cast(uint16_t, lo);
}
// The halves that the values of X are given as in a mode.
template <int MODE>
constexpr int kHalves = MODE == kDown || MODE == kToken ? 2 : 1;

// Adapters of rows as they come, up to this rank: each thread adds those of its own
// outputs by fp32 fma, all of B requested at once.  Above, one adapter after the
// other on the matrix cores: 40 rows of 64 adapters of rank 32 on 6144 x 4096 took
// 24.7 us so and 20.4 by threads, 16 rows 16.4 and 13.6; 512 rows in runs of one
// adapter of rank 16 on 4096 x 4096 61 and 63, in mixed order 72 and 63.
constexpr int kDotRank = 32;

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
  int experts;                    // one row: ids outside [0, experts) are no expert
  const float* weights;           // kDown, kToken
  uint16_t* y16;                  // kSwiglu: h in halves; kLora: Y16 or null
  float* y;                       // kDown: partial rows; kLora: Y or null
  int64_t ldy;
  const int32_t* ids;             // kLora, and one row
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
    const int4 v = a.plan.tiles[y];
    r.e = v.x;
    r.p0 = v.y;
    r.rows = v.z;
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

// 8 entries of one row of A x from the partial sums, in split order; 0 from rp on.
__device__ __forceinline__ void load_t8(const RowsArgs& a, int64_t row, int r, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.f;
  if (r >= a.rp) return;
  const float* p = a.t + row * a.rp + r;
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

// The adapters of 32 rows, added to CB blocks of 32 x 32 sums (MFMA layout:
// lane (c, h), register r: row 8 (r / 4) + 4h + r % 4, column c).  Each adapter
// that stands among the rows is multiplied once for all of them and added to
// its own rows alone; `part` of `parts` callers takes every parts-th adapter.
// A x (fp32) becomes 2^e (high + low fp16 half), both halves exact products
// with B, 64 ranks at a time.  begin() requests A x and the first adapter's B,
// so that a caller can do so before its own loop; add() finishes.
template <int CB>
struct RowAdapters {
  int64_t row;            // the lane's row c in X that has an adapter, or -1
  int id, skip, parts, slot;
  uint32_t all, left, mine;
  int64_t b0[CB];         // the lane's columns of B
  float t[4][8];
  f16x8 bf[CB][4];

  // This caller's next adapter of those left: its slot and rows (0: none).
  __device__ __forceinline__ void next() {
    mine = 0;
    while (left != 0) {
      const int s = __builtin_amdgcn_readlane(id, __builtin_ctz(left));
      const uint32_t m = (uint32_t)__builtin_amdgcn_ballot_w64(row >= 0 && id == s);
      left &= ~m;
      if (skip-- == 0) {
        skip = parts - 1;
        mine = m;
        slot = s;
        return;
      }
    }
  }
  __device__ __forceinline__ void load_t(const RowsArgs& a, int r0) {
#pragma unroll
    for (int q = 0; q < 4; ++q) load_t8(a, row >= 0 ? row : 0, r0 + 16 * q + 8 * (lane_id() >> 5), t[q]);
  }
  // B of the adapter, 64 ranks from r0 on (0 past the rank, where A x is 0 too)
  __device__ __forceinline__ void load_b(const RowsArgs& a, int r0) {
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) {
      const uint16_t* bp = a.b + ((int64_t)slot * a.n + b0[cb]) * a.rank;
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int r = r0 + 16 * q + 8 * (lane_id() >> 5);
        bf[cb][q] = u4_to_f16x8(r < a.rank ? *reinterpret_cast<const uint4*>(bp + r)
                                           : make_uint4(0, 0, 0, 0));
      }
    }
  }
  // xrow: the lane's row c of X, or -1, its id; col[cb]: its column of block cb
  __device__ __forceinline__ void begin(const RowsArgs& a, int64_t xrow, int xid, const int (&col)[CB],
                                        int part, int of) {
    id = xid;
    const bool has = (uint32_t)id < (uint32_t)a.slots;
    row = has ? xrow : -1;
    parts = of;
    skip = part;
    all = left = (uint32_t)__builtin_amdgcn_ballot_w64(has);
#pragma unroll
    for (int cb = 0; cb < CB; ++cb) b0[cb] = min(col[cb], a.n - 1);
    next();
    if (mine == 0) return;
    load_t(a, 0);
    load_b(a, 0);
  }
  __device__ __forceinline__ void add(const RowsArgs& a, f32x16 (&acc)[CB]) {
    if (mine == 0) return;
    const int h = lane_id() >> 5;
    // the rows' powers of two (a lane holds half of its row's entries)
    float top = 0.f;
    for (int r0 = 0; r0 < a.rp; r0 += 64) {
      if (r0 > 0) load_t(a, r0);
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) top = __builtin_fmaxf(top, __builtin_fabsf(t[q][e]));
    }
    const float ts = half_scale(__builtin_fmaxf(top, __shfl_xor(top, 32)));
    const float inv = 1.f / ts;            // a power of two: exact
    float f[16];                           // of the lane's 16 rows
#pragma unroll
    for (int r = 0; r < 16; ++r) f[r] = __shfl(ts, 8 * (r >> 2) + 4 * h + (r & 3));
    const int part = skip;
    for (int r0 = 0; r0 < a.rp; r0 += 64) {
      if (a.rp > 64) load_t(a, r0);
      f16x8 th[4], tl[4];
#pragma unroll
      for (int q = 0; q < 4; ++q)
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float x = t[q][e] * inv;
          th[q][e] = (f16)x;
          tl[q][e] = (f16)(x - (float)th[q][e]);
        }
      const int nq = min(4, (a.rp - r0) / 16);
      const int first = slot;
      const uint32_t first_rows = mine, first_left = left;
      while (true) {
        const uint32_t rows = mine >> (4 * h);   // bit 8 (r / 4) + r % 4: register r's row
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          f32x16 d = {};
#pragma unroll
          for (int q = 0; q < 4; ++q)
            if (q < nq) {
              d = __builtin_amdgcn_mfma_f32_32x32x16_f16(th[q], bf[cb][q], d, 0, 0, 0);
              d = __builtin_amdgcn_mfma_f32_32x32x16_f16(tl[q], bf[cb][q], d, 0, 0, 0);
            }
          if (cb + 1 == CB) {
            // the next adapter's B on its way while this one is added
            next();
            if (mine != 0) load_b(a, r0);
          }
          // (a select, not a product with 0: another row's infinity stays its own)
#pragma unroll
          for (int r = 0; r < 16; ++r) {
            const float with = __builtin_fmaf(f[r], d[r], acc[cb][r]);
            acc[cb][r] = (rows >> (8 * (r >> 2) + (r & 3))) & 1 ? with : acc[cb][r];
          }
        }
        if (mine == 0) break;
      }
      if (r0 + 64 < a.rp) {
        // the next 64 ranks: from the first adapter again
        slot = first;
        mine = first_rows;
        left = first_left;
        skip = part;
        load_b(a, r0 + 64);
      }
    }
  }
};

// --------------------------------------------------- few rows per expert --
// Work-group: up to 32 rows of one expert x 32 CB columns (half or all of a
// 64-row weight tile; kSwiglu: of gate and of up).  Its waves take the K-blocks
// w, w + WAVES, ..., U at a time with every load in flight before the first
// decode, and add their sums in LDS in wave order.  Bound by the latency of the
// few loads between start and sums: 216 pairs over 128 experts of 512 x 1024 at 3
// bits, 38 MB of gate and up fetched (all 128 are 57 MB), take 18 us (2.1 TB/s), their
// down projections at 4 bits 12 us, 40 rows on 6144 x 4096 at 4 bits with adapters 16 us.  More blocks in
// flight (3, 4) changed nothing (16.4, 15.9 us).
// Lane (c, h) supplies X row c / weight row c and K positions 32h + 8s .. +7.
// (Two waves per SIMD at least: with the register file to itself the compiler
// keeps the MFMA results in accumulation registers and copies every one out.)
template <int BITS, int MODE, int WAVES, int CB, int U, bool DOTS>
__global__ __launch_bounds__(WAVES * 64, 2) void k_rows_ksplit(const RowsArgs a) {
  constexpr int WPB = 2 * BITS;
  constexpr int HW = BITS;                   // words of a half block
  constexpr int NM = MODE == kSwiglu ? 2 : 1;
  constexpr int XH = kHalves<MODE>;
  constexpr int PT = CB * 16 / WAVES;        // outputs per thread
  static_assert(CB * 16 % WAVES == 0, "reduction split");
  __shared__ float red[WAVES][CB * 1024];
  const int y = blockIdx.x / a.cols, gx = blockIdx.x % a.cols;
  const int lane = lane_id(), wave = wave_id();
  const int c = lane & 31, h = lane >> 5;
  const int t = CB == 2 ? gx : gx >> 1, cb0 = CB == 2 ? 0 : gx & 1;
  int e = 0, p0 = 32 * y, rows = min(32, a.m - p0);
  if constexpr (MODE != kLora) {
    const int4 v = a.plan.tiles[y];          // (in flight with the number of tiles)
    if (y >= *a.plan.ntiles) return;
    e = v.x;
    p0 = v.y;
    rows = v.z;
  }
  const uint32_t magic = vreg_const(kMagic);
  // uniform: expert e, tile t, columns from cb0 on; a lane: its row of 32
  const int64_t woff = e * a.code_step + ((int64_t)t * a.kb * kTile + 32 * cb0) * WPB;
  const int64_t moff = e * a.meta_step + (int64_t)t * a.G * kTile + 32 * cb0;
  const uint32_t wlane = c * WPB, mlane = c;
  // rows past the tile read its first row (never stored)
  const int64_t xr = x_row<MODE>(a, p0 + (c < rows ? c : 0));
  const uint16_t* xrow = a.X + xr * a.ldx + 32 * h;
  f32x16 acc[NM][CB];
#pragma unroll
  for (int i = 0; i < NM; ++i)
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int r = 0; r < 16; ++r) acc[i][cb][r] = 0.f;
  RowAdapters<CB> adapters;
  int col[CB];
#pragma unroll
  for (int cb = 0; cb < CB; ++cb) col[cb] = t * kTile + 32 * (cb0 + cb) + c;
  // (DOTS) A x of the tile's rows goes to LDS, and every thread adds its own outputs'
  // adapters: their ids, of output p at row out_row(p), column out_col(p)
  constexpr int kDotQ = kDotRank / 8;
  __shared__ f32x4 ts[DOTS ? 32 * 2 * kDotQ : 1];
  auto out_row = [&](int p) __attribute__((always_inline)) {
    const int r = (wave + WAVES * p) & 15;
    return 8 * (r >> 2) + 4 * h + (r & 3);
  };
  auto out_col = [&](int p) __attribute__((always_inline)) {
    return t * kTile + 32 * (cb0 + ((wave + WAVES * p) >> 4)) + c;
  };
  constexpr int TV = MODE == kLora ? (32 * 2 * kDotQ + WAVES * 64 - 1) / (WAVES * 64) : 1;
  f32x4 tv[TV];
  int slot[PT];
  if constexpr (MODE == kLora) {
    if constexpr (DOTS) {
#pragma unroll
      for (int i = 0; i < TV; ++i) {
        // (a row without an adapter has any bits there, and no use for them)
        const int e = threadIdx.x + WAVES * 64 * i, row = e / (2 * kDotQ), r = 4 * (e % (2 * kDotQ));
        tv[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
        if (row < rows && r < a.rp)
          tv[i] = *reinterpret_cast<const f32x4*>(a.t + x_row<MODE>(a, p0 + row) * a.rp + r);
      }
#pragma unroll
      for (int p = 0; p < PT; ++p)
        slot[p] = out_row(p) < rows ? a.ids[x_row<MODE>(a, p0 + out_row(p))] : -1;
    } else {
      adapters.begin(a, c < rows ? xr : -1, c < rows ? a.ids[xr] : -1, col, wave, WAVES);
    }
  }
  for (int jb = wave; jb < a.kb; jb += WAVES * U) {
    f16x8 xa[U][XH][4];
    uint32_t wl[U][NM][CB][HW];
    uint16_t sr[U][NM][CB];
    int zc[U][NM][CB];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int j = min(jb + WAVES * u, a.kb - 1);     // past the range: re-read, not used
      const int64_t g = (a.G == 1) ? 0 : j;
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          const int64_t mi = moff + g * kTile + 32 * cb;
          sr[u][i][cb] = *lane_ptr(a.scale[i], mi, mlane);
          zc[u][i][cb] = *lane_ptr(a.zero[i], mi, mlane);
          load_half<BITS>(lane_ptr(a.codes[i], woff + ((int64_t)j * kTile + 32 * cb) * WPB, wlane), h,
                          wl[u][i][cb]);
        }
      const f16x8* xp = reinterpret_cast<const f16x8*>(xrow + (int64_t)j * (XH * kBlock));
#pragma unroll
      for (int x = 0; x < XH; ++x)
#pragma unroll
        for (int s = 0; s < 4; ++s) xa[u][x][s] = xp[8 * x + s];
    }
    loads_issued();
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (jb + WAVES * u >= a.kb) break;
#pragma unroll
      for (int i = 0; i < NM; ++i)
#pragma unroll
        for (int cb = 0; cb < CB; ++cb) {
          const DeqT<BITS> d = make_deq_b<BITS>(1.f, zc[u][i][cb]);
          f32x16 blk = {};
#pragma unroll
          for (int s = 0; s < 4; ++s) {
            const f16x8 w = int_half<BITS>(wl[u][i][cb], s, d, magic);
#pragma unroll
            for (int x = 0; x < XH; ++x)
              blk = __builtin_amdgcn_mfma_f32_32x32x16_f16(xa[u][x][s], w, blk, 0, 0, 0);
          }
          const float sc = h2f(sr[u][i][cb]);
#pragma unroll
          for (int r = 0; r < 16; ++r) acc[i][cb][r] = __builtin_fmaf(sc, blk[r], acc[i][cb][r]);
        }
    }
  }
  constexpr int PC = PT < 4 ? PT : 4;        // outputs whose B is requested together
  uint4 bq[PC][kDotQ];
  auto request_b = [&](int p1) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PC; ++i) {
      const bool has = (uint32_t)slot[p1 + i] < (uint32_t)a.slots && out_col(p1 + i) < a.n;
      const uint16_t* b = a.b + (has ? ((int64_t)slot[p1 + i] * a.n + out_col(p1 + i)) * a.rank : 0);
#pragma unroll
      for (int q = 0; q < kDotQ; ++q)
        if (8 * q < a.rank) bq[i][q] = *reinterpret_cast<const uint4*>(b + 8 * q);
    }
  };
  if constexpr (MODE == kLora) {
    if constexpr (DOTS) {
#pragma unroll
      for (int i = 0; i < TV; ++i) {
        const int e = threadIdx.x + WAVES * 64 * i;
        if (e < 32 * 2 * kDotQ) ts[e] = tv[i];
      }
      request_b(0);
    } else {
      adapters.add(a, acc[0]);
    }
  }
  // thread (wave, lane) finishes registers wave, wave + WAVES, ... of the CB x 16
  float v[NM][PT];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    if (i > 0) __syncthreads();
#pragma unroll
    for (int cb = 0; cb < CB; ++cb)
#pragma unroll
      for (int r = 0; r < 16; ++r) red[wave][1024 * cb + 64 * r + lane] = acc[i][cb][r];
    __syncthreads();
#pragma unroll
    for (int p = 0; p < PT; ++p) {
      float sum = red[0][64 * (wave + WAVES * p) + lane];
#pragma unroll
      for (int w = 1; w < WAVES; ++w) sum += red[w][64 * (wave + WAVES * p) + lane];
      v[i][p] = sum;
    }
  }
  if constexpr (MODE == kLora) {
    if constexpr (DOTS) {
#pragma unroll
      for (int p1 = 0; p1 < PT; p1 += PC) {
        if (p1 > 0) request_b(p1);
#pragma unroll
        for (int i = 0; i < PC; ++i) {
          float s = 0.f;
#pragma unroll
          for (int q = 0; q < kDotQ; ++q) {
            if (8 * q >= a.rank) continue;
            const f32x4 x = ts[2 * kDotQ * out_row(p1 + i) + 2 * q], y = ts[2 * kDotQ * out_row(p1 + i) + 2 * q + 1];
            const f16x8 b = u4_to_f16x8(bq[i][q]);
#pragma unroll
            for (int e = 0; e < 4; ++e) s = __builtin_fmaf(x[e], (float)b[e], s);
#pragma unroll
            for (int e = 0; e < 4; ++e) s = __builtin_fmaf(y[e], (float)b[4 + e], s);
          }
          if ((uint32_t)slot[p1 + i] < (uint32_t)a.slots) v[0][p1 + i] += s;
        }
      }
    }
  }
#pragma unroll
  for (int p = 0; p < PT; ++p) {
    const int cl = out_col(p), row = out_row(p);
    if (row >= rows || cl >= a.n) continue;
    if constexpr (MODE == kSwiglu) {
      put_halves(a.y16 + (int64_t)(p0 + row) * a.ldy, cl, silu(v[0][p]) * v[1][p]);
    } else if constexpr (MODE == kDown) {
      const int64_t pair = a.plan.order[p0 + row];
      a.y[pair * a.ldy + cl] = a.weights[pair] * v[0][p];
    } else {
      const int64_t o = x_row<MODE>(a, p0 + row) * a.ldy + cl;
      if (a.y != nullptr) a.y[o] = v[0][p];
      if (a.y16 != nullptr) a.y16[o] = __builtin_bit_cast(uint16_t, (f16)v[0][p]);
    }
  }
}

// ---------------------------------------------------------------- one row --
// Work-group: 64 / NG outputs of one (token, slot) pair (kSwiglu, from gate and
// up) or of one token (kToken: the K-blocks of all its slots, each with its own
// row of h, its own weights and its weight beside the group's scale).  Lane NG r
// + g: weight row r, slice g of every block, decoded and multiplied by vector
// dot products: with one row of X the matrix cores would be idle in 31 of 32
// rows, and few outputs per work-group spread even a small product over all CUs
// (the 2048 outputs of a token's down projections: 14.3 us as 64 work-groups of
// 32 columns; now 6.5 us, and 7.8 us for gate and up of 8 experts of 1024 x 2048 at
// 4 bits, 18.4 MB).  Bound by launch latency and one round of loads.
template <int BITS, int MODE, int NG, int WAVES, int U>
__global__ __launch_bounds__(WAVES * 64) void k_rows_gemv(const RowsArgs a) {
  constexpr int WPB = 2 * BITS;
  constexpr int RW = 64 / NG;                // outputs per work-group
  constexpr int XQ = 8 / NG;                 // 16-byte chunks of x per slice
  constexpr int XH = kHalves<MODE>;
  constexpr int NM = MODE == kSwiglu ? 2 : 1;
  constexpr int SW = SliceWords<BITS, NG>::n;
  __shared__ float red[NM][WAVES][RW];
  const uint32_t magic = vreg_const(kMagic);
  const int lane = lane_id(), wave = wave_id();
  const int r = lane / NG, g = lane % NG;
  const int y = blockIdx.x / a.cols, gx = blockIdx.x % a.cols;
  const int t = gx / NG, r0 = RW * (gx % NG);
  int e = 0;
  if constexpr (MODE == kSwiglu) {
    e = a.ids[y];
    if ((uint32_t)e >= (uint32_t)a.experts) return;
  }
  const int64_t woff = ((int64_t)t * a.kb * kTile + r0) * WPB, moff = (int64_t)t * a.G * kTile + r0;
  float acc[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) acc[i] = 0.f;
  // K-blocks j0, j0 + step, ... of one row of x by one expert's weights
  auto product = [&](int ex, const uint16_t* xrow, float f, int j0, int step) __attribute__((always_inline)) {
    const int64_t wo = ex * a.code_step + woff, mo = ex * a.meta_step + moff;
    for (int jb = j0; jb < a.kb; jb += step * U) {
      uint32_t wd[U][NM][SW];
      uint16_t sr[U][NM];
      int zc[U][NM];
      uint4 xv[U][XH][XQ];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int j = min(jb + step * u, a.kb - 1);        // past the range: re-read, not used
        const int64_t mi = mo + (a.G == 1 ? 0 : j) * (int64_t)kTile;
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          load_slice_words<BITS, NG>(lane_ptr(a.codes[i], wo + (int64_t)j * kTile * WPB, r * WPB), g,
                                     wd[u][i]);
          sr[u][i] = *lane_ptr(a.scale[i], mi, r);
          zc[u][i] = *lane_ptr(a.zero[i], mi, r);
        }
        const uint4* xp =
            reinterpret_cast<const uint4*>(lane_ptr(xrow, (int64_t)j * (XH * kBlock), 8 * XQ * g));
#pragma unroll
        for (int x = 0; x < XH; ++x)
#pragma unroll
          for (int q = 0; q < XQ; ++q) xv[u][x][q] = xp[8 * x + q];
      }
      loads_issued();
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (jb + step * u >= a.kb) break;
        f16x2 xs[XH][4 * XQ];
#pragma unroll
        for (int x = 0; x < XH; ++x)
#pragma unroll
          for (int q = 0; q < XQ; ++q) {
            xs[x][4 * q] = as_h2(xv[u][x][q].x);
            xs[x][4 * q + 1] = as_h2(xv[u][x][q].y);
            xs[x][4 * q + 2] = as_h2(xv[u][x][q].z);
            xs[x][4 * q + 3] = as_h2(xv[u][x][q].w);
          }
#pragma unroll
        for (int i = 0; i < NM; ++i) {
          const float s = MODE == kToken ? f * h2f(sr[u][i]) : h2f(sr[u][i]);
          float dot = slice_dot<BITS, NG>(wd[u][i], xs[0], zc[u][i], g, magic);
          if constexpr (XH == 2) dot += slice_dot<BITS, NG>(wd[u][i], xs[1], zc[u][i], g, magic);
          acc[i] = __builtin_fmaf(s, dot, acc[i]);
        }
      }
    }
  };
  if constexpr (MODE == kSwiglu) {
    product(e, a.X + (int64_t)(y / a.top_k) * a.ldx, 1.f, wave, WAVES);
  } else {
    // `parts` waves per slot share its K-blocks (more slots than waves: in turn)
    const int parts = max(1, WAVES / a.top_k);
    for (int s = wave / parts; s < a.top_k; s += WAVES / parts) {
      const int64_t pair = (int64_t)y * a.top_k + s;
      const int ex = a.ids[pair];
      if ((uint32_t)ex >= (uint32_t)a.experts) continue;
      product(ex, a.X + pair * a.ldx, a.weights[pair], wave % parts, parts);
    }
  }
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    acc[i] = slice_sum<NG>(acc[i]);
    if (g == 0) red[i][wave][r] = acc[i];
  }
  lds_barrier();
  if (wave != 0 || lane >= RW) return;
  float tot[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    tot[i] = red[i][0][lane];
#pragma unroll
    for (int w = 1; w < WAVES; ++w) tot[i] += red[i][w][lane];
  }
  const int col = t * kTile + r0 + lane;     // (n % 64 == 0)
  if constexpr (MODE == kSwiglu) {
    put_halves(a.y16 + (int64_t)y * a.ldy, col, silu(tot[0]) * tot[1]);
  } else {
    const int64_t o = (int64_t)y * a.ldy + col;
    if (a.y != nullptr) a.y[o] = tot[0];
    if (a.y16 != nullptr) a.y16[o] = __builtin_bit_cast(uint16_t, (f16)tot[0]);
  }
}

// Keeps the compiler from moving the computation of v past this point.
__device__ __forceinline__ void here(f16x8& v) { asm volatile("" : "+v"(v)); }

// -------------------------------------------------- many rows per expert --
// Work-group: 64 rows of one expert x 256 columns, 4 waves of 64 rows x 64
// columns: tile 4x + w (kSwiglu: 32 columns of gate and the same 32 of up, half
// w % 2 of tile 2x + w / 2).  A wave decodes its two 32-column blocks straight
// into MFMA B registers -- integers q - z, exact, no scale rounded into them --
// and multiplies them by both 32-row blocks of X, read from LDS once for the
// two (16-byte chunks permuted within their row by xswz, so that the reads fall
// on distinct banks).  The four MFMAs of 32 x 32 outputs and a K-block start
// from 0, and the group's scale takes their sum to the fp32 accumulators: 16 fma
// per lane, laid beside the next four MFMAs with a quarter of the next decode.
// X by direct-to-LDS loads into four stages, three blocks ahead (and the next
// block's first operands are read before the barrier), codes two blocks ahead in
// registers; one barrier per block.
// Two halves of X (kDown) lie in a stage one behind the other; the low ones of a product
// are read beside the MFMAs of its high ones into registers of their own (a second set of
// those spills 12 registers at 4 bits, 22 at 8).
// Bound by instruction issue: 205 vector instructions beside 16 MFMAs a block, of
// them 64 the scaling and 72 decoding (4 bits); one issues in 92 % of the cycles of
// 16384 pairs through 32 experts of 2 x 1408 x 2048 (212 to 273 us over 12 calls, 890 to
// 690 TFLOP/s; MFMA busy 48 %).  In their down projections, 32 MFMAs a block (191 to 226
// us), one issues in 70 % and the matrix cores are busy in 58 %: the chains of eight
// MFMAs on one block of sums, with 22 K-blocks only.  2048
// rows on 4096 x 4096 without adapters: 78 us, 64 of them in the loop.  128 rows x
// 128 columns (130 vector instructions a block, twice the operand reads) took 81
// us there, as this form did then, and 359 for 331 us over 64 experts of 256 rows; two waves a
// work-group 402 for 386 us.
// Codes, scales and zeros come through buffer descriptors: the base and the
// block's offset are scalars, so a load costs no vector address, neither the
// instructions that form one nor the registers that a loop keeps one in (48
// bytes per lane for the six pointers of two matrices).
using Buffer = __amdgpu_buffer_rsrc_t;
__device__ __forceinline__ Buffer buffer_of(const void* p, int64_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc(const_cast<void*>(p), 0, (int)bytes, 0x00020000);
}
// 16 bytes per lane to LDS, lane l's to lds + 16 l.
__device__ __forceinline__ void buffer_to_lds(Buffer b, void* lds, uint32_t lane, int at) {
  typedef __attribute__((address_space(3))) void lds_void;
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)lds, 16, lane, at, 0, 0);
}
// load_half through a descriptor: the words of half h of a row of 64 codes.
// lane = half_offsets(): where its first (BITS < 5: all) and its high plane's lie.
template <int BITS>
__device__ __forceinline__ int2 half_offsets(int c, int h) {
  constexpr int high = BITS == 5 ? 4 : BITS == 6 ? 8 : 12;
  const int row = 8 * BITS * c;
  if constexpr (BITS >= 5 && BITS <= 7) return make_int2(row + 16 * h, row + 32 + high * h);
  else return make_int2(row + 4 * BITS * h, 0);
}
template <int BITS>
__device__ __forceinline__ void load_half(Buffer b, int2 lane, int at, uint32_t* wl) {
  auto put = [&](auto v, int n, uint32_t* w) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < n; ++i) w[i] = v[i];
  };
  if constexpr (BITS == 2) {
    put(__builtin_amdgcn_raw_buffer_load_b64(b, lane.x, at, 0), 2, wl);
  } else if constexpr (BITS == 3) {
    put(__builtin_amdgcn_raw_buffer_load_b96(b, lane.x, at, 0), 3, wl);
  } else {
    put(__builtin_amdgcn_raw_buffer_load_b128(b, lane.x, at, 0), 4, wl);
    if constexpr (BITS == 5) wl[4] = __builtin_amdgcn_raw_buffer_load_b32(b, lane.y, at, 0);
    if constexpr (BITS == 6) put(__builtin_amdgcn_raw_buffer_load_b64(b, lane.y, at, 0), 2, wl + 4);
    if constexpr (BITS == 7) put(__builtin_amdgcn_raw_buffer_load_b96(b, lane.y, at, 0), 3, wl + 4);
    if constexpr (BITS == 8) put(__builtin_amdgcn_raw_buffer_load_b128(b, lane.x + 16, at, 0), 4, wl + 4);
  }
}

// X stages: LDS objects of their own, so that the compiler can tell which
// direct-to-LDS loads a read depends on.
constexpr int kXStages = 4;
template <int I, int XH>
__device__ __forceinline__ f16x8* x_stage() {
  __shared__ f16x8 xs[XH * 64 * 8];
  return xs;
}

// Waits for the wave's LDS accesses and for all but its N newest loads, then a
// work-group barrier.  (One asm block: a fence, as in lds_barrier(), would wait
// for every direct-to-LDS load in flight.)
template <int N>
__device__ __forceinline__ void stage_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(N) : "memory");
}

template <int BITS, int MODE>
__global__ __launch_bounds__(256, 2) void k_rows_tiled(const RowsArgs a) {
  constexpr int WPB = 2 * BITS;
  constexpr int HW = BITS;
  constexpr int XH = kHalves<MODE>;
  const RowTile rt = row_tile<MODE>(a, 64);
  if (rt.rows <= 0) return;
  const int gx = rt.col;
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  const int c = lane & 31, h = lane >> 5;
  const uint32_t magic = vreg_const(kMagic);
  const int tiles = (a.n + kTile - 1) / kTile;
  const int tile = MODE == kSwiglu ? 2 * gx + (wave >> 1) : 4 * gx + wave;
  // column block f: rows 32 half[f] of the tile (kSwiglu: of matrix f)
  const int half[2] = {MODE == kSwiglu ? wave & 1 : 0, MODE == kSwiglu ? wave & 1 : 1};
  const int dt = min(tile, tiles - 1);       // (a tile past the matrix: its last one, never stored)
  const int64_t woff = rt.e * a.code_step + (int64_t)dt * a.kb * kTile * WPB;
  const int64_t moff = rt.e * a.meta_step + (int64_t)dt * a.G * kTile;
  constexpr int NM = MODE == kSwiglu ? 2 : 1;
  Buffer codes[NM], scale[NM], zero[NM];
#pragma unroll
  for (int i = 0; i < NM; ++i) {
    codes[i] = buffer_of(a.codes[i] + woff, (int64_t)a.kb * kTile * WPB * 4);
    scale[i] = buffer_of(a.scale[i] + moff, (int64_t)a.G * kTile * 2);
    zero[i] = buffer_of(a.zero[i] + moff, (int64_t)a.G * kTile);
  }
  const int2 wlane = half_offsets<BITS>(c, h);
  // Direct-to-LDS loads of X: instruction i of a wave brings 8 rows from row
  // 32 i + 8 wave on, lane l to chunk l of the 64: row l / 8, slot l % 8.  32-bit
  // offsets: from the first row of kDown's consecutive ones, else from X, whose
  // span the host has checked (tiled_form).
  const Buffer xbuf = buffer_of(a.X + (MODE == kDown ? rt.p0 * a.ldx : 0), 0xffffffff);
  uint32_t xoff[2];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int r = 32 * i + (tid >> 3), p = r < rt.rows ? r : 0;
    const int64_t row = MODE == kDown ? p : x_row<MODE>(a, rt.p0 + p);
    xoff[i] = (uint32_t)(row * a.ldx + 8 * xswz(r, tid & 7)) * 2;
  }

  uint32_t wl[2][2][HW];                    // [slot][block]
  uint16_t sr[2][2];
  int zc[2][2];
  auto request_x = [&](auto T, int j) __attribute__((always_inline)) {
    f16x8* xs = x_stage<decltype(T)::value, XH>();
    const int jj = min(j, a.kb - 1);
#pragma unroll
    for (int x = 0; x < XH; ++x)
#pragma unroll
      for (int i = 0; i < 2; ++i)
        buffer_to_lds(xbuf, xs + 512 * x + 256 * i + 64 * wave, xoff[i], (XH * jj + x) * kBlock * 2);
    __builtin_amdgcn_sched_barrier(0);
  };
  auto request_w = [&](auto S, int j) __attribute__((always_inline)) {
    constexpr int u = decltype(S)::value;
    const int jj = min(j, a.kb - 1);
    const int g = (a.G == 1) ? 0 : jj;
#pragma unroll
    for (int f = 0; f < 2; ++f) {
      const int i = min(f, NM - 1);
      load_half<BITS>(codes[i], wlane, (jj * kTile + 32 * half[f]) * WPB * 4, wl[u][f]);
      sr[u][f] = __builtin_amdgcn_raw_buffer_load_b16(scale[i], 2 * c, 2 * (g * kTile + 32 * half[f]), 0);
      zc[u][f] = __builtin_amdgcn_raw_buffer_load_b8(zero[i], c, g * kTile + 32 * half[f], 0);
    }
  };
  f32x16 acc[2][2], blk[2];                // [row block][column block]; sums not yet scaled
  f16x8 av[2][4], bv[2][4];                  // [row / column block][K quarter]
  f16x8 al[4];                               // (two halves) the low ones of the next product
  float scl[2];                              // the scales of bv's operands
  auto read_a = [&](auto R, auto T) __attribute__((always_inline)) {
    constexpr int rb = decltype(R)::value;
    const f16x8* xs = x_stage<decltype(T)::value, XH>();
#pragma unroll
    for (int q = 0; q < 4; ++q) av[rb][q] = xs[8 * (32 * rb + c) + xswz(c, 4 * h + q)];
  };
  auto read_low = [&](auto R, auto T) __attribute__((always_inline)) {
    constexpr int rb = decltype(R)::value;
    if constexpr (XH == 2) {
      const f16x8* xs = x_stage<decltype(T)::value, XH>() + 512;
#pragma unroll
      for (int q = 0; q < 4; ++q) al[q] = xs[8 * (32 * rb + c) + xswz(c, 4 * h + q)];
    }
  };
  const std::integral_constant<int, 0> I0;
  const std::integral_constant<int, 1> I1;
  const std::integral_constant<int, 2> I2;
  const std::integral_constant<int, 3> I3;
  // quarters q0 .. q1 - 1 of column block F from slot S
  auto decode = [&](auto S, auto F, int q0, int q1) __attribute__((always_inline)) {
    constexpr int u = decltype(S)::value, f = decltype(F)::value;
    const DeqT<BITS> d = make_deq_b<BITS>(1.f, zc[u][f]);
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      if (q < q0 || q >= q1) continue;
      bv[f][q] = int_half<BITS>(wl[u][f], q, d, magic);
      here(bv[f][q]);
    }
  };
  auto scale_of = [&](auto S, auto F) __attribute__((always_inline)) {
    constexpr int u = decltype(S)::value, f = decltype(F)::value;
    float s = h2f(sr[u][f]);
    asm volatile("" : "+v"(s));
    return s;
  };
  // the MFMAs (four for each half) of row block R and column block F into blk[R]
  auto product = [&](auto R, auto F) __attribute__((always_inline)) {
    constexpr int rb = decltype(R)::value, f = decltype(F)::value;
    const f32x16 none = {};
#pragma unroll
    for (int q = 0; q < 4; ++q)
      blk[rb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(av[rb][q], bv[f][q], q == 0 ? none : blk[rb],
                                                       0, 0, 0);
    if constexpr (XH == 2) {
#pragma unroll
      for (int q = 0; q < 4; ++q)
        blk[rb] = __builtin_amdgcn_mfma_f32_32x32x16_f16(al[q], bv[f][q], blk[rb], 0, 0, 0);
    }
  };
  // those sums, times s, to the accumulators
  auto scaled = [&](auto R, auto F, float s) __attribute__((always_inline)) {
    constexpr int rb = decltype(R)::value, f = decltype(F)::value;
#pragma unroll
    for (int r = 0; r < 16; ++r) acc[rb][f][r] = __builtin_fmaf(s, blk[rb][r], acc[rb][f][r]);
  };
  request_x(I0, 0);
  request_w(I0, 0);
  request_x(I1, 1);
  request_w(I1, 1);
  request_x(I2, 2);
#pragma unroll
  for (int r = 0; r < 16; ++r) {
    acc[0][0][r] = acc[0][1][r] = acc[1][0][r] = acc[1][1][r] = 0.f;
    blk[1][r] = 0.f;
  }
  scl[1] = 0.f;
  decode(I0, I0, 0, 4);
  scl[0] = scale_of(I0, I0);
  stage_barrier<0>();
  read_a(I0, I0);
  read_low(I0, I0);
  // loads of a wave and a block behind the one that must be there: X's of the
  // next block and the codes', scales' and zeros' issued after it
  constexpr int kNewer = 2 * XH + 2 * ((BITS >= 5 ? 2 : 1) + 2);
  // Block j, its codes in slot j % 2, its rows in stage j % 4 = T; block j + 3's
  // rows go where block j - 1's were.
  auto step = [&](auto T, int j) __attribute__((always_inline)) {
    constexpr int kT = decltype(T)::value;
    const std::integral_constant<int, kT % 2> U;
    const std::integral_constant<int, (kT + 1) % 2> N;
    const std::integral_constant<int, (kT + 1) % kXStages> T1;
    const std::integral_constant<int, (kT + 3) % kXStages> T3;
    request_x(T3, j + 3);
    read_a(I1, T);
    __builtin_amdgcn_sched_barrier(0);
    product(I0, I0);
    scaled(I1, I1, scl[1]);                  // of block j - 1
    decode(U, I1, 0, 2);
    __builtin_amdgcn_sched_barrier(0);
    read_low(I1, T);
    product(I1, I0);
    decode(U, I1, 2, 4);
    scl[1] = scale_of(U, I1);
    scaled(I0, I0, scl[0]);
    __builtin_amdgcn_sched_barrier(0);
    read_low(I0, T);
    request_w(U, j + 2);
    product(I0, I1);
    decode(N, I0, 0, 2);
    scaled(I1, I0, scl[0]);
    __builtin_amdgcn_sched_barrier(0);
    read_low(I1, T);
    read_a(I0, T1);                          // (of block j + 1)
    product(I1, I1);
    decode(N, I0, 2, 4);
    scl[0] = scale_of(N, I0);
    scaled(I0, I1, scl[1]);
    __builtin_amdgcn_sched_barrier(0);
    read_low(I0, T1);
    stage_barrier<kNewer>();                 // block j + 2's rows are there
  };
  int j0 = 0;
  for (; j0 + 4 <= a.kb; j0 += 4) {
    step(I0, j0);
    step(I1, j0 + 1);
    step(I2, j0 + 2);
    step(I3, j0 + 3);
  }
  if (j0 < a.kb) step(I0, j0);
  if (j0 + 1 < a.kb) step(I1, j0 + 1);
  if (j0 + 2 < a.kb) step(I2, j0 + 2);
  stage_barrier<0>();                        // (rows requested past the end)
  scaled(I1, I1, scl[1]);

  int col[2];
#pragma unroll
  for (int f = 0; f < 2; ++f) col[f] = tile * kTile + 32 * half[f] + c;
  if constexpr (MODE == kLora) {
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      const int64_t row = 32 * rb + c < rt.rows ? x_row<MODE>(a, rt.p0 + 32 * rb + c) : -1;
      RowAdapters<2> adapters;
      adapters.begin(a, row, row >= 0 ? a.ids[row] : -1, col, 0, 1);
      adapters.add(a, acc[rb]);
    }
  }
  if constexpr (MODE == kSwiglu) {
    if (tile >= tiles) return;
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        const int at = 32 * rb + 8 * (r >> 2) + 4 * h + (r & 3);
        if (at >= rt.rows) continue;
        put_halves(a.y16 + (int64_t)(rt.p0 + at) * a.ldy, col[0],
                   silu(acc[rb][0][r]) * acc[rb][1][r]);
      }
  } else {
    // lane c's row c of each row block: its output row and weight, read together
    // and handed to the lanes that store it
    int out[2];
    float w[2] = {1.f, 1.f};
#pragma unroll
    for (int rb = 0; rb < 2; ++rb) {
      const int p = rt.p0 + (32 * rb + c < rt.rows ? 32 * rb + c : 0);
      out[rb] = MODE == kDown ? a.plan.order[p] : (int)x_row<MODE>(a, p);
    }
    if constexpr (MODE == kDown) {
#pragma unroll
      for (int rb = 0; rb < 2; ++rb) w[rb] = a.weights[out[rb]];
    }
#pragma unroll
    for (int rb = 0; rb < 2; ++rb)
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        if constexpr (MODE == kDown) {
          const int at = 8 * (r >> 2) + 4 * h + (r & 3);
          const int64_t y0 = (int64_t)__shfl(out[rb], at) * a.ldy;
          const float ws = __shfl(w[rb], at);
          if (32 * rb + at >= rt.rows) continue;
#pragma unroll
          for (int f = 0; f < 2; ++f)
            if (col[f] < a.n) a.y[y0 + col[f]] = ws * acc[rb][f][r];
        } else {
          // A register of either column block holds rows R and R + 4 in the wave's
          // halves: with the inner halves swapped, each is 64 columns of one row,
          // a whole line of fp16 (81 -> 77 us for 2048 rows on 4096 x 4096; fp32 rows
          // of the experts, two half lines a store as they are, lost by it: 145 -> 165).
          const float x = acc[rb][0][r], y = acc[rb][1][r];
          const auto v = __builtin_amdgcn_permlane32_swap(__builtin_bit_cast(uint32_t, x),
                                                          __builtin_bit_cast(uint32_t, y), false, false);
          const int cl = tile * kTile + lane;
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const int at = 8 * (r >> 2) + (r & 3) + 4 * i;
            if (32 * rb + at >= rt.rows) continue;
            const int64_t o = (int64_t)__builtin_amdgcn_readlane(out[rb], at) * a.ldy + cl;
            const uint32_t bits = v[i];
            const float s = __builtin_bit_cast(float, bits);
            if (cl >= a.n) continue;
            if (a.y != nullptr) a.y[o] = s;
            if (a.y16 != nullptr) a.y16[o] = __builtin_bit_cast(uint16_t, (f16)s);
          }
        }
      }
  }
}

}  // namespace qlin
