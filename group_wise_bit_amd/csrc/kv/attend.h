// Attention of one new token per sequence over the cache (gfx950, wave64).
#pragma once

#include "kv_layout.h"

namespace qlin {

constexpr int kAttendWaves = 4;
constexpr int kAttendRows = 16;        // query heads of a work-group: a column block of an MFMA

struct AttendArgs {
  KvSeqs s;
  const uint8_t* data;
  int64_t head_bytes;        // bytes of a page of one head
  const f16* q;
  int64_t ldq;
  float* o;
  f16* o16;
  int64_t ldo;
  float* lse;
  float* part;               // [2 work-groups][rows][D]: sums of cut sequences
  float* stat;               // [2 work-groups][rows][2]: their offset and weight
  int heads, kv_heads, ratio;
  int rows;                  // query heads per work-group, min(ratio, 16)
  int rts;                   // work-groups' row blocks per head of the cache
  int window, groups;
  float c;                   // scale * log2(e)
};

// Tokens [lo, hi) that a sequence sees.
__device__ __forceinline__ void seen_tokens(const AttendArgs& a, int b, int& lo, int& hi) {
  const int len = max(a.s.lengths[b], 0);
  const int room = a.s.width * (kKvTile << a.s.page_log);
  lo = a.window > 0 ? max(len - a.window, 0) : 0;
  hi = min(len, room);
}
__device__ __forceinline__ int seen_tiles(const AttendArgs& a, int b) {
  int lo, hi;
  seen_tokens(a, b, lo, hi);
  return hi > lo ? (hi + kKvTile - 1) / kKvTile - lo / kKvTile : 0;
}

// Tiles of all sequences before b = `until`, or all.
__device__ __forceinline__ int64_t tiles_before(const AttendArgs& a, int until) {
  const int lane = lane_id();
  int64_t total = 0;
  for (int base = 0; base < until; base += 64) {
    const int n = base + lane < until ? seen_tiles(a, base + lane) : 0;
    total += __builtin_amdgcn_readlane(scan64(n), 63);
  }
  return total;
}

// Every work-group takes `share` tiles of the list [sequence][head][row block][tile].
__device__ __forceinline__ int64_t tile_share(int64_t all, int groups) {
  const int64_t s = (all + groups - 1) / groups;
  return s < kAttendWaves ? kAttendWaves : s;
}

template <int D, int KB, int VB>
struct KvRegs {
  static constexpr int G = D / 64;
  u32x4 k[KB * G / 4], v[VB * G / 4];
  u32x4 ks[G], vs[G];
  uint32_t kz[(G + 1) / 2];
  u32x2 vz[G];
};

template <int D, int KB, int VB>
__device__ __forceinline__ void load_tile(KvRegs<D, KB, VB>& t, const uint8_t* p) {
  using T = KvTile<D, KB, VB>;
  constexpr int G = D / 64;
  const int lane = lane_id(), g = lane >> 4, r = lane & 15;
#pragma unroll
  for (int i = 0; i < KB * G / 4; ++i) t.k[i] = *(const u32x4*)(p + T::k + (i * 64 + lane) * 16);
  if constexpr (KB < 16) {
#pragma unroll
    for (int c = 0; c < G; ++c) t.ks[c] = *(const u32x4*)(p + T::ks + c * 64 + g * 16);
    if constexpr (G == 1) t.kz[0] = *(const uint16_t*)(p + T::kz + r * 2);
    if constexpr (G == 2) t.kz[0] = *(const uint32_t*)(p + T::kz + r * 4);
    if constexpr (G == 4) {
      const u32x2 z = *(const u32x2*)(p + T::kz + r * 8);
      t.kz[0] = z[0];
      t.kz[1] = z[1];
    }
  }
#pragma unroll
  for (int i = 0; i < VB * G / 4; ++i) t.v[i] = *(const u32x4*)(p + T::v + (i * 64 + lane) * 16);
  if constexpr (VB < 16) {
#pragma unroll
    for (int c = 0; c < G; ++c) {
      t.vs[c] = *(const u32x4*)(p + T::vs + c * 64 + g * 16);
      t.vz[c] = *(const u32x2*)(p + T::vz + (g * G + c) * 8);
    }
  }
}

// Pairs of codes as fp16 numbers q - z, exactly: the code's bits go into the mantissa of
// 1024 (bits 0..3 or 0..7) or, 16 times larger, of 1024 with a factor 1/16.
// c1 = -(1024 + z) of the pair's two zero points, c2 = -(64 + z).
__device__ __forceinline__ f16x2 code_low(uint32_t w, uint32_t mask, uint32_t magic, f16x2 c1) {
  return as_h2((w & mask) | magic) + c1;
}
__device__ __forceinline__ f16x2 code_high(uint32_t w, uint32_t mask, uint32_t magic, f16x2 c2) {
  return __builtin_elementwise_fma(as_h2((w & mask) | magic), f16x2{(f16)0.0625f, (f16)0.0625f}, c2);
}
// -(1024 + z) of two bytes of w.
template <int B0, int B1>
__device__ __forceinline__ f16x2 zero_pair(uint32_t w) {
  return as_h2(__builtin_amdgcn_perm(0xE4E4E4E4u, w, 0x04000400u | (B1 << 16) | B0));
}

__device__ __forceinline__ float max16x32(float v) {     // over lanes l, l ^ 16, l ^ 32, l ^ 48
  v = fmaxf(v, __shfl_xor(v, 16));
  return fmaxf(v, __shfl_xor(v, 32));
}
__device__ __forceinline__ float sum16x32(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// The running state of a wave for 16 query heads: lane (g, n) = (l / 16, l % 16) has the
// sums of head n for dims 64 c + 16 g + 4 i + j in o[c][j][i], and the weight l of its
// own tokens.  All are relative to 2^off.
template <int D>
struct AttendState {
  static constexpr int G = D / 64;
  f32x4 o[G][4];
  float l, m, off;
  int e;                     // exponent of the largest scale of values so far (uniform)
};

// A tile of 32 tokens.  Keys are the rows of the first products' A operand and query
// heads its columns, so that S comes out with head n of a lane's tokens 4 g + i
// of each half -- the order in which the second products' B operand wants P, with values as the rows of A:
// no data crosses lanes but the maximum.  Scales of keys multiply the sums of a
// group; scales of values multiply P, which enters as two fp16 halves (hi rounded
// towards zero, lo the rest: 21 bits).  So that P * s has these bits whatever the
// size of s, P is taken relative to 2^off, off = max + e - 15, s < 2^e for every scale
// so far: P s < 2^15.
template <int D, int KB, int VB>
__device__ __forceinline__ void attend_tile(AttendState<D>& st, KvRegs<D, KB, VB>& t,
                                            const f16x8 (&q)[D / 32], float c, bool edge, int first,
                                            int lo, int hi, uint32_t magic) {
  constexpr int G = D / 64;
  const int lane = lane_id(), g = lane >> 4;
  constexpr uint32_t klow = KB == 4 ? 0x000F000Fu : 0x00FF00FFu;
  constexpr uint32_t vlow = VB == 4 ? 0x000F000Fu : 0x00FF00FFu;
  float x[8];
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    f32x4 acc[G];
#pragma unroll
    for (int cg = 0; cg < G; ++cg) {
      f16x2 c1{}, c2{};
      if constexpr (KB < 16) {
        const int byte = h * G + cg;
        const uint32_t sel = 0x04000400u | ((byte % 4) << 16) | (byte % 4);
        c1 = as_h2(__builtin_amdgcn_perm(0xE4E4E4E4u, t.kz[byte / 4], sel));
        if constexpr (KB == 4) c2 = c1 + f16x2{(f16)960.f, (f16)960.f};
      }
      f32x4 s{};
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        union { f16x8 v; f16x2 p[4]; uint32_t w[4]; } f;
        const int at = (h * G + cg) * (KB / 2) + u * (KB / 4);      // word of the lane's run
        if constexpr (KB == 4) {
          const uint32_t w = t.k[at / 4][at % 4], w8 = w >> 8;
          f.p[0] = code_low(w, klow, magic, c1);
          f.p[1] = code_high(w, klow << 4, magic, c2);
          f.p[2] = code_low(w8, klow, magic, c1);
          f.p[3] = code_high(w8, klow << 4, magic, c2);
        } else if constexpr (KB == 8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = t.k[(at + i) / 4][(at + i) % 4];
            f.p[2 * i] = code_low(w, klow, magic, c1);
            f.p[2 * i + 1] = code_low(w >> 8, klow, magic, c1);
          }
        } else {
          f.v = __builtin_bit_cast(f16x8, t.k[at / 4]);
        }
        s = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.v, q[cg * 2 + u], s, 0, 0, 0);
      }
      acc[cg] = s;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float s = 0.f;
#pragma unroll
      for (int cg = 0; cg < G; ++cg) {
        if constexpr (KB < 16) {
          const f16x2 sc = as_h2(t.ks[cg][h * 2 + i / 2]);
          s = __builtin_fmaf(acc[cg][i], (float)sc[i % 2], s);
        } else {
          s += acc[cg][i];
        }
      }
      x[h * 4 + i] = s * c;
    }
  }
  if (edge) {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int p = first + (i >> 2) * 16 + 4 * g + (i & 3);
      const bool in = p >= lo && p < hi;
      if (!in) {
        x[i] = -__builtin_inff();
        // (what lies there may be no number, and 0 times that is none either)
        if constexpr (VB < 16) {
#pragma unroll
          for (int cg = 0; cg < G; ++cg) t.vs[cg][i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        } else {
#pragma unroll
          for (int b = 0; b < 4 * G; ++b) t.v[b][i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        }
      }
    }
  }
  float mx = x[0];
#pragma unroll
  for (int i = 1; i < 8; ++i) mx = fmaxf(mx, x[i]);
  st.m = fmaxf(st.m, max16x32(mx));
  if constexpr (VB < 16) {
    // the largest scale of the tile: fp16 patterns of one sign are ordered as integers
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    u16x2 top{};
#pragma unroll
    for (int cg = 0; cg < G; ++cg)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint32_t pair = t.vs[cg][i];
        top = __builtin_elementwise_max(top, __builtin_bit_cast(u16x2, pair));
      }
    const int one = max((int)top[0], (int)top[1]);
    int all = __builtin_amdgcn_readlane(one, 0);
    all = max(all, __builtin_amdgcn_readlane(one, 16));
    all = max(all, __builtin_amdgcn_readlane(one, 32));
    all = max(all, __builtin_amdgcn_readlane(one, 48));
    st.e = max(st.e, (all >> 10) - 14);
  }
  const float off = st.m + (float)(st.e - 15);
  if (__ballot(off != st.off) != 0) {
    const float f = __builtin_amdgcn_exp2f(st.off - off);
    st.l *= f;
#pragma unroll
    for (int cg = 0; cg < G; ++cg)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[cg][j] *= f;
    st.off = off;
  }
  float p[8];
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    p[i] = __builtin_amdgcn_exp2f(x[i] - off);
    st.l += p[i];
  }
  union { f16x8 v; f16x2 p[4]; } ph, pl;
#pragma unroll
  for (int cg = 0; cg < G; ++cg) {
    if (VB < 16 || cg == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float w0 = p[2 * i], w1 = p[2 * i + 1];
        if constexpr (VB < 16) {
          const f16x2 sc = as_h2(t.vs[cg][i]);
          w0 *= (float)sc[0];
          w1 *= (float)sc[1];
        }
        ph.p[i] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(w0, w1));
        pl.p[i] = __builtin_bit_cast(
            f16x2, __builtin_amdgcn_cvt_pkrtz(w0 - (float)ph.p[i][0], w1 - (float)ph.p[i][1]));
      }
    }
    f16x2 c1[4], c2[4];
    if constexpr (VB < 16) {
      c1[0] = zero_pair<0, 1>(t.vz[cg][0]);
      c1[1] = zero_pair<2, 3>(t.vz[cg][0]);
      c1[2] = zero_pair<0, 1>(t.vz[cg][1]);
      c1[3] = zero_pair<2, 3>(t.vz[cg][1]);
      if constexpr (VB == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c2[i] = c1[i] + f16x2{(f16)960.f, (f16)960.f};
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      union { f16x8 v; f16x2 p[4]; } f;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (VB == 4) {
          const uint32_t w = j < 2 ? t.v[cg][i] : t.v[cg][i] >> 8;
          f.p[i] = j % 2 == 0 ? code_low(w, vlow, magic, c1[i]) : code_high(w, vlow << 4, magic, c2[i]);
        } else if constexpr (VB == 8) {
          const uint32_t w = t.v[cg * 2 + j / 2][i];
          f.p[i] = code_low(j % 2 == 0 ? w : w >> 8, vlow, magic, c1[i]);
        } else {
          f.p[i] = as_h2(t.v[cg * 4 + j][i]);
        }
      }
      st.o[cg][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.v, ph.v, st.o[cg][j], 0, 0, 0);
      st.o[cg][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.v, pl.v, st.o[cg][j], 0, 0, 0);
    }
  }
}

// The table entries of 64 pages, one per lane.
struct PageList {
  int base, entry;
};

template <int D, int KB, int VB>
__global__ __launch_bounds__(256) void k_attend(const AttendArgs a) {
  using T = KvTile<D, KB, VB>;
  constexpr int G = D / 64;
  constexpr int kPad = 4;                // a row's pitch in LDS is not a multiple of the banks
  __shared__ float red[kAttendWaves][kAttendRows][D + kPad];
  __shared__ float rst[kAttendWaves][kAttendRows][2];
  const int lane = lane_id(), wave = wave_id(), g = lane >> 4, n = lane & 15;
  const uint32_t magic = vreg_const(kMagic);
  const int hgs = a.kv_heads * a.rts;
  const int64_t all = tiles_before(a, a.s.seqs) * hgs;
  const int64_t share = tile_share(all, a.groups);
  const int64_t from = blockIdx.x * share, to = min(from + share, all);
  if (from >= to) return;
  // the sequence that tile `from` belongs to
  int b = 0, tiles = 0;
  int64_t at = 0;                        // first tile of (b, head 0)
  for (int base = 0; base < a.s.seqs; base += 64) {
    const int t = base + lane < a.s.seqs ? seen_tiles(a, base + lane) : 0;
    const int sum = scan64(t);
    const uint64_t past = __ballot(at + (int64_t)sum * hgs > from);
    if (past != 0) {
      const int l = __builtin_ctzll(past);
      b = base + l;
      tiles = __builtin_amdgcn_readlane(t, l);
      at += (int64_t)(__builtin_amdgcn_readlane(sum, l) - tiles) * hgs;
      break;
    }
    at += (int64_t)__builtin_amdgcn_readlane(sum, 63) * hgs;
  }
  int hg = (int)((from - at) / tiles);
  int64_t begin = at + (int64_t)hg * tiles;      // first tile of (b, hg)
  int64_t pos = from;
  while (pos < to) {
    int lo, hi;
    seen_tokens(a, b, lo, hi);
    const int tile0 = lo / kKvTile;
    const int head = hg / a.rts, row0 = (hg % a.rts) * kAttendRows;
    const int rows = min(a.ratio - row0, kAttendRows);
    const int first = tile0 + (int)(pos - begin);
    const int last = tile0 + (int)(min(to, begin + tiles) - begin);
    // ---- this wave's tiles: first + wave, first + wave + 4, ...
    const int qh = head * a.ratio + row0 + min(n, rows - 1);
    f16x8 q[D / 32];
    const f16* qp = a.q + b * a.ldq + (int64_t)qh * D;
#pragma unroll
    for (int i = 0; i < D / 32; ++i) {
      const f16x8 z = {};
      const f16x8 v = *(const f16x8*)(qp + (i / 2) * 64 + g * 16 + (i % 2) * 8);
      q[i] = n < rows ? v : z;
    }
    AttendState<D> st;
#pragma unroll
    for (int c = 0; c < G; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[c][j] = f32x4{};
    st.l = 0.f;
    st.m = -1e30f;
    st.off = -1e30f;
    st.e = VB < 16 ? -14 : 0;
    const int32_t* row = a.s.table + b * a.s.ld;
    PageList pages{-64, 0};
    for (int t = first + wave; t < last; t += kAttendWaves) {
      const int pi = t >> a.s.page_log;
      if (pi - pages.base >= 64) {
        pages.base = pi;
        pages.entry = pi + lane < a.s.width ? row[pi + lane] : -1;
      }
      const int page = __builtin_amdgcn_readlane(pages.entry, pi - pages.base);
      if (page < 0 || page >= a.s.pages) continue;
      const uint8_t* tp = a.data + ((int64_t)page * a.kv_heads + head) * a.head_bytes +
                          (t & ((1 << a.s.page_log) - 1)) * T::bytes;
      KvRegs<D, KB, VB> regs;
      load_tile<D, KB, VB>(regs, tp);
      const int p0 = t * kKvTile;
      attend_tile<D, KB, VB>(st, regs, q, a.c, p0 < lo || p0 + kKvTile > hi, p0, lo, hi, magic);
    }
    st.l = sum16x32(st.l);
    // ---- the waves' sums together
    if (g == 0) {
      rst[wave][n][0] = st.off;
      rst[wave][n][1] = st.l;
    }
    lds_barrier();
    float off = rst[0][n][0];
#pragma unroll
    for (int w = 1; w < kAttendWaves; ++w) off = fmaxf(off, rst[w][n][0]);
    const float f = __builtin_amdgcn_exp2f(st.off - off);
#pragma unroll
    for (int c = 0; c < G; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int i = 0; i < 4; ++i) red[wave][n][c * 64 + g * 16 + 4 * i + j] = st.o[c][j][i] * f;
    lds_barrier();
    const bool cut_front = pos > begin, cut_back = to < begin + tiles;
    const bool cut = cut_front || cut_back;
    const int64_t slot = 2 * (int64_t)blockIdx.x + (cut_front ? 0 : 1);
    for (int i = threadIdx.x; i < rows * (D / 4); i += 256) {
      const int r = i / (D / 4), d = i % (D / 4) * 4;
      float m = rst[0][r][0];
#pragma unroll
      for (int w = 1; w < kAttendWaves; ++w) m = fmaxf(m, rst[w][r][0]);
      float l = 0.f;
      f32x4 v{};
#pragma unroll
      for (int w = 0; w < kAttendWaves; ++w) {
        l += rst[w][r][1] * __builtin_amdgcn_exp2f(rst[w][r][0] - m);
        v += *(const f32x4*)&red[w][r][d];
      }
      const int h = head * a.ratio + row0 + r;
      if (cut) {
        *(f32x4*)(a.part + (slot * a.rows + r) * D + d) = v;
        if (d == 0) {
          a.stat[(slot * a.rows + r) * 2] = m;
          a.stat[(slot * a.rows + r) * 2 + 1] = l;
        }
      } else {
        v *= l == 0.f ? 0.f : 1.f / l;
        const int64_t out = b * a.ldo + (int64_t)h * D + d;
        if (a.o != nullptr) *(f32x4*)(a.o + out) = v;
        if (a.o16 != nullptr) {
          typedef f16 f16x4 __attribute__((ext_vector_type(4)));
          *(f16x4*)(a.o16 + out) = f16x4{(f16)v[0], (f16)v[1], (f16)v[2], (f16)v[3]};
        }
        if (a.lse != nullptr && d == 0)
          a.lse[(int64_t)b * a.heads + h] =
              l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994531f;
      }
    }
    lds_barrier();                       // (the next segment writes red and rst again)
    pos = min(to, begin + tiles);
    if (pos >= to) break;
    begin += tiles;
    if (++hg == hgs) {
      hg = 0;
      do { tiles = seen_tiles(a, ++b); } while (tiles == 0);
    }
  }
}

// The parts of the sequences that more than one work-group dealt with, and rows without
// tokens.  One work-group per (sequence, query head): its waves take the parts in turn.
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(const AttendArgs a) {
  constexpr int V = D / 64;              // dims per lane
  __shared__ float red[4][D];
  __shared__ float rst[4][2];
  const int lane = lane_id(), wave = wave_id();
  const int b = blockIdx.x, h = blockIdx.y;
  const int hgs = a.kv_heads * a.rts;
  const int tiles = seen_tiles(a, b);
  const int kvh = h / a.ratio, r16 = h % a.ratio;
  const int hg = kvh * a.rts + r16 / kAttendRows, r = r16 % kAttendRows;
  float o[V] = {}, l = 0.f, m = -1e30f;
  if (tiles > 0) {
    const int64_t before = tiles_before(a, b), all = tiles_before(a, a.s.seqs) * hgs;
    const int64_t share = tile_share(all, a.groups);
    const int64_t begin = before * hgs + (int64_t)hg * tiles, end = begin + tiles;
    const int64_t w0 = begin / share, w1 = (end - 1) / share;
    if (w0 == w1) return;                // one work-group had all of it
    for (int64_t w = w0 + wave; w <= w1; w += 4) {
      const int64_t at = (2 * w + (begin < w * share ? 0 : 1)) * a.rows + r;
      const float pm = a.stat[at * 2], pl = a.stat[at * 2 + 1];
      const float nm = fmaxf(m, pm);
      const float f = __builtin_amdgcn_exp2f(m - nm), pf = __builtin_amdgcn_exp2f(pm - nm);
      l = l * f + pl * pf;
      m = nm;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] = o[i] * f + a.part[at * D + lane + 64 * i] * pf;
    }
    if (lane == 0) {
      rst[wave][0] = m;
      rst[wave][1] = l;
    }
#pragma unroll
    for (int i = 0; i < V; ++i) red[wave][lane + 64 * i] = o[i];
  }
  __syncthreads();
  if (wave != 0) return;
  if (tiles > 0) {
    float top = rst[0][0];
    for (int w = 1; w < 4; ++w) top = fmaxf(top, rst[w][0]);
    l = 0.f;
    for (int i = 0; i < V; ++i) o[i] = 0.f;
    for (int w = 0; w < 4; ++w) {
      const float f = __builtin_amdgcn_exp2f(rst[w][0] - top);
      l += rst[w][1] * f;
#pragma unroll
      for (int i = 0; i < V; ++i) o[i] += red[w][lane + 64 * i] * f;
    }
    m = top;
  }
  const float inv = l == 0.f ? 0.f : 1.f / l;
#pragma unroll
  for (int i = 0; i < V; ++i) {
    const int64_t out = b * a.ldo + (int64_t)h * D + lane + 64 * i;
    if (a.o != nullptr) a.o[out] = o[i] * inv;
    if (a.o16 != nullptr) a.o16[out] = (f16)(o[i] * inv);
  }
  if (a.lse != nullptr && lane == 0)
    a.lse[(int64_t)b * a.heads + h] =
        l == 0.f ? -__builtin_inff() : (m + __builtin_log2f(l)) * 0.69314718055994531f;
}

}  // namespace qlin
