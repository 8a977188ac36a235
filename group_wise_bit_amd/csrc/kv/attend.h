// Attention of one new token per sequence over the cache (gfx950, wave64):
//     S[p] = scale q . k_p,   P = exp(S - max),   O = sum P v_p / sum P,
// in one pass over the cached tokens with running sums and a unit of them; k = s (code - z).
//
// What bounds it.  Every code is read once for up to 16 query heads and takes part in 4 ratio
// operations, far below what the matrix cores do, so that the bytes of the cache are the floor.  With 8
// bits and more they are reached (64 sequences of 8192 tokens, 8 heads of 128: 196 us for 1.13 GB, 5.7
// TB/s).  With 4 bits a tile of 32 tokens and 128 dims takes 383 vector instructions of a wave, 24 of
// them MFMAs (prologue and sums of the waves included): 131071 tokens of 8 heads take 39 us (3.8
// TB/s), 20 of them issue (at 2.4 GHz), 28 their bytes; a wave waits for its loads and results a third
// of its cycles and for an issue slot another third, at three waves a SIMD.  A ragged batch (48
// sequences of 1 to 4096 tokens, 28.8 us, 12 of issue, 15 of bytes) is bound by the starts of its 384
// row blocks: about five tiles a wave, each start a page list, queries, a first tile and three
// barriers with nothing in flight.
//
// Why this split.  One query head per sequence and head of the cache is no matrix product:
// the heads that share a head of the cache (ratio, up to 16 at a time) are one MFMA operand, tokens
// are the other.  A wave takes every fourth tile of its work-group's range, so that no barrier
// is in the loop.  The tiles of all sequences are one list, cut into equal ranges for as many
// work-groups as the chip holds: a batch of 48 lengths from 1 to 4096 and one sequence of
// 131071 tokens both fill it.
#pragma once

#include "kv_layout.h"

namespace qlin {

typedef float f32x2 __attribute__((ext_vector_type(2)));

constexpr int kAttendWaves = 4;
constexpr int kAttendRows = 16;        // query heads of a work-group: a column block of an MFMA
constexpr int kMaxParts = 1024;        // work-groups at most, and parts of a sequence
constexpr float kNoScore = -1e30f;     // a running maximum of none: below every finite score

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
  float* stat;               // [2 work-groups][rows][2]: the score they are relative to, their weight
  int heads, kv_heads, ratio;
  int rows;                  // query heads per work-group, min(ratio, 16)
  int rts;                   // work-groups' row blocks per head of the cache
  int window, groups;
  bool whole;                // a work-group per sequence and row block, nothing to join
  uint32_t flip;             // sign bits of a negative scale
  float c;                   // |scale| * log2(e), above 0
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

// Every work-group takes `share` units of the list [sequence][head][row block][units]:
// kStartUnits for the start of a row block's tiles, then one for each of them.  (A start costs
// a page list, the queries, the sums of four waves and a store.  48 sequences of 1 to 4096 tokens:
// 51 us without, 30.4 with 4 units, 29.2 with 8, 30.1 with 16.)  The least share is a tile for every
// wave: few tokens are a chain of a wave's loads, and the join has time for the parts (9 windows of
// 1000 tokens, 256 dims of 16 bits: 10.4 us for 13.0 with 12 units, one sequence of 4000, 128
// dims of 4 bits: 8.7 for 10.0; with their joins 15.4 for 17.1 and 14.0 for 15.9).  A range may lie
// within a start's units: it has no tiles then, and no place among the parts.
constexpr int kStartUnits = 8;
__device__ __forceinline__ int seen_units(const AttendArgs& a, int b) {
  const int tiles = seen_tiles(a, b);
  return tiles > 0 ? tiles + kStartUnits : 0;
}
__device__ __forceinline__ int64_t unit_share(int64_t all, int groups) {
  const int64_t s = (all + groups - 1) / groups;
  return s < kAttendWaves ? kAttendWaves : s;
}

// A tile in registers, as it lies in memory: a wave's loads are whole 16-byte units.  (Through
// LDS, with direct-to-LDS loads in two stages, four work-groups per CU instead of three: the same
// on 48 sequences of 4096 tokens and 4 bits, 33.2 us with the join; slower on one of 131071,
// 44.5 : 42.5, and on 64 of 8192 with 8 bits, 203 : 198.  With three stages 35 us for 29 of the first.)
template <int D, int KB, int VB>
struct KvRegs {
  static constexpr int G = D / 64;
  u32x4 k[KB * G / 4], v[VB * G / 4];
  u32x4 ks[G], vs[G];
  uint32_t kz[(G + 1) / 2];
  u32x2 vz[G];

  __device__ __forceinline__ void load(const uint8_t* p) {
    using T = KvTile<D, KB, VB>;
    const int lane = lane_id(), g = lane >> 4, r = lane & 15;
#pragma unroll
    for (int i = 0; i < KB * G / 4; ++i) k[i] = *(const u32x4*)(p + T::k + (i * 64 + lane) * 16);
    if constexpr (KB < 16) {
#pragma unroll
      for (int c = 0; c < G; ++c) ks[c] = *(const u32x4*)(p + T::ks + c * 64 + g * 16);
      if constexpr (G == 1) kz[0] = *(const uint16_t*)(p + T::kz + r * 2);
      if constexpr (G == 2) kz[0] = *(const uint32_t*)(p + T::kz + r * 4);
      if constexpr (G == 4) {
        const u32x2 z = *(const u32x2*)(p + T::kz + r * 8);
        kz[0] = z[0];
        kz[1] = z[1];
      }
    }
#pragma unroll
    for (int i = 0; i < VB * G / 4; ++i) v[i] = *(const u32x4*)(p + T::v + (i * 64 + lane) * 16);
    if constexpr (VB < 16) {
#pragma unroll
      for (int c = 0; c < G; ++c) {
        vs[c] = *(const u32x4*)(p + T::vs + c * 64 + g * 16);
        vz[c] = *(const u32x2*)(p + T::vz + (g * G + c) * 8);
      }
    }
  }
};

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

// Constants that the compiler does not know: a * x + b of an fp16 number x with these is
// one v_fma_mix_f32, where a product or a difference would first convert x.
struct MixConsts {
  uint32_t magic;
  float zero, minus;
};
__device__ __forceinline__ MixConsts mix_consts() {
  return MixConsts{vreg_const(kMagic), __builtin_bit_cast(float, vreg_const(0u)),
                   __builtin_bit_cast(float, vreg_const(0xBF800000u))};
}

__device__ __forceinline__ float max16x32(float v) {     // over lanes l, l ^ 16, l ^ 32, l ^ 48
  const uint32_t x = __builtin_bit_cast(uint32_t, v);
  const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  v = fmaxf(__builtin_bit_cast(float, (uint32_t)a[0]), __builtin_bit_cast(float, (uint32_t)a[1]));
  const uint32_t y = __builtin_bit_cast(uint32_t, v);
  const auto b = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return fmaxf(__builtin_bit_cast(float, (uint32_t)b[0]), __builtin_bit_cast(float, (uint32_t)b[1]));
}
__device__ __forceinline__ float sum16x32(float v) {
  v += __shfl_xor(v, 16);
  return v + __shfl_xor(v, 32);
}

// The running state of a wave for 16 query heads: lane (g, n) = (l / 16, l % 16) has the
// sums of head n for dims 64 c + 16 g + 4 i + j in o[c][j][i], and the weight l of its
// own tokens.  A token of score x weighs p = 2^((x - r) c + k).
template <int D>
struct AttendState {
  static constexpr int G = D / 64;
  f32x4 o[G][4];
  float l, r, k;
};

// A tile of 32 tokens.  Keys are the rows of the first products' A operand and query
// heads its columns, so that S comes out with head n of a lane's tokens 4 g + i
// of each half -- the order in which the second products' B operand wants P, with values as the rows of A:
// no data crosses lanes but the maximum.  Scales of keys multiply the sums of a
// group; scales of values multiply P, which enters as two fp16 halves (hi rounded
// towards zero, lo the rest to nearest: 22 bits, and no side that all roundings go to).  So that
// P * s has these bits whatever the sizes of s and of P where s is large, p is taken in units in
// which the largest p s so far is 2^14 to 2^16 (an s below 2^-24, fp16's least number, counts as that, so that weights stay below
// 2^40): where a p s reaches 2^16, k falls, and where it does by far (with the first tile of a
// wave, say), r rises to the largest score.  As long as none does, no lane needs to know of
// another's scores.  Exponents are formed from differences of scores, which fp32 holds whatever
// their size (from 2^24 on a rounding of r c alone would be 1 or more).
constexpr float kRoom = 0x1p16f;
constexpr float kFar = 0x1p64f;        // p s from here on, and k below kLeast: r is taken anew, too
constexpr float kLeast = -32.f;
constexpr float kUnset = 1000.f;       // k of no token: the first weight is beyond any room
template <int D, int KB, int VB>
__device__ __forceinline__ void attend_tile(AttendState<D>& st, const KvRegs<D, KB, VB>& t,
                                            const f16x8 (&q)[D / 32], float c, bool edge, int first,
                                            int lo, int hi, MixConsts mix) {
  constexpr int G = D / 64;
  const uint32_t magic = mix.magic;
  constexpr int kUnits = KB * G / 4, kHalf = kUnits >= 2 ? kUnits / 2 : 1;
  const int lane = lane_id(), g = lane >> 4;
  constexpr uint32_t klow = KB == 4 ? 0x000F000Fu : 0x00FF00FFu;
  constexpr uint32_t vlow = VB == 4 ? 0x000F000Fu : 0x00FF00FFu;
  float x[8];
  u32x4 ks[G];
  if constexpr (KB < 16) {
#pragma unroll
    for (int cg = 0; cg < G; ++cg) ks[cg] = t.ks[cg];
  }
  u32x4 ku[kHalf];                       // the half tile's units
#pragma unroll
  for (int h = 0; h < 2; ++h) {
    if (h == 0 || kUnits >= 2) {
#pragma unroll
      for (int i = 0; i < kHalf; ++i) ku[i] = t.k[h * kHalf + i];
    }
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
        // word of the lane's run, from its half's first unit on
        const int at = (h * G + cg) * (KB / 2) + u * (KB / 4) - (kUnits >= 2 ? h * kHalf * 4 : 0);
        if constexpr (KB == 4) {
          const uint32_t w = ku[at / 4][at % 4], w8 = w >> 8;
          f.p[0] = code_low(w, klow, magic, c1);
          f.p[1] = code_high(w, klow << 4, magic, c2);
          f.p[2] = code_low(w8, klow, magic, c1);
          f.p[3] = code_high(w8, klow << 4, magic, c2);
        } else if constexpr (KB == 8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = ku[(at + i) / 4][(at + i) % 4];
            f.p[2 * i] = code_low(w, klow, magic, c1);
            f.p[2 * i + 1] = code_low(w >> 8, klow, magic, c1);
          }
        } else {
          f.v = __builtin_bit_cast(f16x8, ku[at / 4]);
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
          const f16x2 sc = as_h2(ks[cg][h * 2 + i / 2]);
          s = __builtin_fmaf(acc[cg][i], (float)sc[i % 2], s);
        } else {
          s += acc[cg][i];
        }
      }
      x[h * 4 + i] = s;
    }
  }
  u32x4 vs[G];
  u32x4 mask{~0u, ~0u, ~0u, ~0u};        // (16 bits) of the seen tokens' values
  if constexpr (VB < 16) {
#pragma unroll
    for (int cg = 0; cg < G; ++cg) vs[cg] = t.vs[cg];
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
          for (int cg = 0; cg < G; ++cg) vs[cg][i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        } else {
          mask[i / 2] &= i % 2 ? 0x0000FFFFu : 0xFFFF0000u;
        }
      }
    }
  }
  // the largest scale of a token's groups (a NaN is passed over)
  uint32_t top[4];
  if constexpr (VB < 16) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      top[i] = 0x00010001u;
#pragma unroll
      for (int cg = 0; cg < G; ++cg) top[i] = pk_max(top[i], vs[cg][i]);
    }
  }
  float p[8];
  // the weights, and the largest p s of the lane's tokens
  auto weigh = [&](float r, float k) {
    float most = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      p[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(x[i] - r, c, k));
      most = fmaxf(most, VB < 16 ? __builtin_fmaf((float)as_h2(top[i / 2])[i % 2], p[i], mix.zero) : p[i]);
    }
    return most;
  };
  float most = weigh(st.r, st.k);
  if (__ballot(most >= kRoom) != 0) {
    most = max16x32(most);
    float r = st.r, k = fminf(st.k, st.k + (float)(15 - __builtin_amdgcn_frexp_expf(most))), to = k - st.k;
    if (__ballot(most >= kFar || k < kLeast) != 0) {
      r = x[0];
#pragma unroll
      for (int i = 1; i < 8; ++i) r = fmaxf(r, x[i]);
      r = fmaxf(st.r, max16x32(r));
      // (a tile whose weights are all 0 leaves k as it is)
      most = fmaxf(max16x32(weigh(r, 0.f)), 0x1p-126f);
      k = fminf(__builtin_fmaf(r - st.r, c, st.k), (float)(15 - __builtin_amdgcn_frexp_expf(most)));
      // (above 40 only for a head without scores so far, whose p are 0)
      to = fminf(k, 41.f);
    }
    const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(st.r - r, c, k - st.k));
    to = __builtin_amdgcn_exp2f(to);
#pragma unroll
    for (int i = 0; i < 8; ++i) p[i] *= to;
    st.l *= f;
#pragma unroll
    for (int cg = 0; cg < G; ++cg)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[cg][j] *= f;
    st.r = r;
    st.k = k;
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) st.l += p[i];
  union { f16x8 v; f16x2 p[4]; } ph, pl;
#pragma unroll
  for (int cg = 0; cg < G; ++cg) {
    if (VB < 16 || cg == 0) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        float w0 = p[2 * i], w1 = p[2 * i + 1];
        if constexpr (VB < 16) {
          const uint32_t pair = vs[cg][i];
          w0 = __builtin_fmaf((float)as_h2(pair)[0], w0, mix.zero);
          w1 = __builtin_fmaf((float)as_h2(pair)[1], w1, mix.zero);
        }
        ph.p[i] = __builtin_bit_cast(f16x2, __builtin_amdgcn_cvt_pkrtz(w0, w1));
        pl.p[i] = __builtin_convertvector(
            (f32x2{__builtin_fmaf((float)ph.p[i][0], mix.minus, w0),
                   __builtin_fmaf((float)ph.p[i][1], mix.minus, w1)}), f16x2);
      }
    }
    f16x2 c1[4], c2[4];
    if constexpr (VB < 16) {
      const u32x2 z = t.vz[cg];
      c1[0] = zero_pair<0, 1>(z[0]);
      c1[1] = zero_pair<2, 3>(z[0]);
      c1[2] = zero_pair<0, 1>(z[1]);
      c1[3] = zero_pair<2, 3>(z[1]);
      if constexpr (VB == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i) c2[i] = c1[i] + f16x2{(f16)960.f, (f16)960.f};
      }
    }
    u32x4 vu{};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      union { f16x8 v; f16x2 p[4]; } f;
      if (j % (16 / VB) == 0) {
        const int unit = cg * (VB / 4) + j / (16 / VB);
        vu = t.v[unit];
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if constexpr (VB == 4) {
          const uint32_t w = j < 2 ? vu[i] : vu[i] >> 8;
          f.p[i] = j % 2 == 0 ? code_low(w, vlow, magic, c1[i]) : code_high(w, vlow << 4, magic, c2[i]);
        } else if constexpr (VB == 8) {
          const uint32_t w = vu[i];
          f.p[i] = code_low(j % 2 == 0 ? w : w >> 8, vlow, magic, c1[i]);
        } else {
          f.p[i] = as_h2(vu[i] & mask[i]);
        }
      }
      st.o[cg][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.v, ph.v, st.o[cg][j], 0, 0, 0);
      st.o[cg][j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(f.v, pl.v, st.o[cg][j], 0, 0, 0);
    }
  }
}

__device__ __forceinline__ f16x8 signed_by(f16x8 v, uint32_t flip) {
  return __builtin_bit_cast(f16x8, __builtin_bit_cast(u32x4, v) ^ flip);
}

// The table entries of 64 pages, one per lane.
struct PageList {
  int base, entry;
};

// Two tiles of a wave in registers, one loading while the other is used; or one, where
// two gain nothing: 128 dims of 16 bits 47.8 us : 48.2 with one, 256 dims of 8 bits 43.3 : 40.1, of
// 16 bits 50.1 : 48.2 (48 sequences of 1 to 4096 tokens; the other waves' loads are enough there).
constexpr bool attend_two(int d, int kb, int vb) { return d <= 128 && (kb + vb) * (d / 64) <= 32; }
// Work-groups per CU that the grid and the registers are sized for (four waves each, one per SIMD).
// Small tiles three: 168 registers, 3 of them spilled (16 bytes of scratch a lane) with 128 dims of 4
// bits; two take 30.3 us for 27.8 (48 sequences, 128 dims, 4 bits), four with one tile 29.2; 64 dims
// 12.2 (three) : 13.0 (four).  256 dims with up to 16 bits together two: 4 bits 28.8 for 37.3 with one,
// 8 bits 36.0 for 40.1 (13 registers spilled; more bits do not fit).  The others two, or one: 64
// and 128 dims with a side of 16 bits have registers for one more, which is not measured.  Every
// instance spills 17 to 35 scalar registers to lanes of vector ones.
constexpr int attend_occupancy(int d, int kb, int vb) {
  return d == 256 ? (kb + vb <= 16 ? 2 : 1) : (kb + vb) * (d / 64) <= 16 ? 3 : 2;
}

template <int D, int KB, int VB>
__global__ __launch_bounds__(256, attend_occupancy(D, KB, VB)) void k_attend(
    const AttendArgs a) {
  using T = KvTile<D, KB, VB>;
  constexpr int G = D / 64;
  constexpr int kRow = D + 4;            // a row's pitch in LDS is not a multiple of the banks
  __shared__ float rst[kAttendWaves][kAttendRows][2];
  __shared__ float red[2 * kAttendRows * kRow];      // sums of two waves
  const int lane = lane_id(), wave = wave_id(), g = lane >> 4, n = lane & 15;
  const MixConsts mix = mix_consts();
  const int hgs = a.kv_heads * a.rts;
  int b = 0, hg = 0, units = 0;          // of (b, hg)
  int64_t begin = 0, pos = 0, to = 0;    // where these begin, and the work-group's own
  if (a.whole) {
    b = blockIdx.x / hgs;
    hg = blockIdx.x % hgs;
    units = seen_units(a, b);
    to = units;
    if (units == 0) {
      const int row0 = hg / a.rts * a.ratio + hg % a.rts * kAttendRows;
      const int rows = min(a.ratio - hg % a.rts * kAttendRows, kAttendRows);
      for (int i = threadIdx.x; i < rows * D; i += 256) {
        const int64_t out = b * a.ldo + (int64_t)row0 * D + i;
        if (a.o != nullptr) a.o[out] = 0.f;
        if (a.o16 != nullptr) a.o16[out] = (f16)0.f;
      }
      if (a.lse != nullptr && threadIdx.x < (unsigned)rows)
        a.lse[(int64_t)b * a.heads + row0 + threadIdx.x] = -__builtin_inff();
      return;
    }
  } else {
    // the sequence that this work-group's first unit belongs to
    const int t0 = lane < a.s.seqs ? seen_units(a, lane) : 0;
    const int sum0 = scan64(t0);
    int64_t all = __builtin_amdgcn_readlane(sum0, 63);
    for (int base = 64; base < a.s.seqs; base += 64) {
      const int t = base + lane < a.s.seqs ? seen_units(a, base + lane) : 0;
      all += __builtin_amdgcn_readlane(scan64(t), 63);
    }
    all *= hgs;
    const int64_t share = unit_share(all, a.groups);
    pos = blockIdx.x * share;
    to = min(pos + share, all);
    if (pos >= to) return;
    for (int base = 0; base < a.s.seqs; base += 64) {
      const int t = base == 0 ? t0 : base + lane < a.s.seqs ? seen_units(a, base + lane) : 0;
      const int sum = base == 0 ? sum0 : scan64(t);
      const uint64_t past = __ballot(begin + (int64_t)sum * hgs > pos);
      if (past != 0) {
        const int l = __builtin_ctzll(past);
        b = base + l;
        units = __builtin_amdgcn_readlane(t, l);
        begin += (int64_t)(__builtin_amdgcn_readlane(sum, l) - units) * hgs;
        break;
      }
      begin += (int64_t)__builtin_amdgcn_readlane(sum, 63) * hgs;
    }
    hg = (int)((pos - begin) / units);
    begin += (int64_t)hg * units;
  }
  for (;;) {
    int lo, hi;
    seen_tokens(a, b, lo, hi);
    const int tile0 = lo / kKvTile;
    const int head = hg / a.rts, row0 = (hg % a.rts) * kAttendRows;
    const int rows = min(a.ratio - row0, kAttendRows);
    // own tiles of the row block (none, if the range ends with the start's units)
    const int64_t tiles0 = begin + kStartUnits;
    const int first = tile0 + (int)(max(pos, tiles0) - tiles0);
    const int last = tile0 + (int)(min(to, begin + units) - tiles0);
    if (first >= last) break;
    AttendState<D> st;
#pragma unroll
    for (int c = 0; c < G; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[c][j] = f32x4{};
    st.l = 0.f;
    st.r = kNoScore;
    st.k = kUnset;
    // ---- this wave's tiles: first + wave, first + wave + 4, ...
    int t = first + wave;
    if (t < last) {
      const int32_t* row = a.s.table + b * a.s.ld;
      PageList pages{-64, 0};
      // where tile t lies (somewhere, if its page is not there)
      bool there[2];
      auto place = [&](int t, bool& ok) {
        const int pi = t >> a.s.page_log;
        if (pi - pages.base >= 64) {
          pages.base = pi;
          pages.entry = pi + lane < a.s.width ? row[pi + lane] : -1;
        }
        const int page = __builtin_amdgcn_readlane(pages.entry, pi - pages.base);
        ok = page >= 0 && page < a.s.pages;
        return a.data + ((int64_t)(ok ? page : 0) * a.kv_heads + head) * a.head_bytes +
               (t & ((1 << a.s.page_log) - 1)) * T::bytes;
      };
      const uint8_t* tp = place(t, there[0]);
      KvRegs<D, KB, VB> one;
      one.load(tp);
      f16x8 q[D / 32];
      const f16* qp = a.q + b * a.ldq + (int64_t)(head * a.ratio + row0 + min(n, rows - 1)) * D;
#pragma unroll
      for (int i = 0; i < D / 32; ++i) {
        const f16x8 z = {};
        const f16x8 v = *(const f16x8*)(qp + (i / 2) * 64 + g * 16 + (i % 2) * 8);
        q[i] = n < rows ? signed_by(v, a.flip) : z;
      }
      auto use = [&](const auto& tile, int t) {
        const int p0 = t * kKvTile;
        attend_tile<D, KB, VB>(st, tile, q, a.c, p0 < lo || p0 + kKvTile > hi, p0, lo, hi, mix);
      };
      if constexpr (attend_two(D, KB, VB)) {
        KvRegs<D, KB, VB> two;
        for (;;) {
          two.load(place(min(t + kAttendWaves, last - 1), there[1]));
          if (there[0]) use(one, t);
          t += kAttendWaves;
          if (t >= last) break;
          one.load(place(min(t + kAttendWaves, last - 1), there[0]));
          if (there[1]) use(two, t);
          t += kAttendWaves;
          if (t >= last) break;
        }
      } else {
        for (;;) {
          if (there[0]) use(one, t);
          t += kAttendWaves;
          if (t >= last) break;
          one.load(place(t, there[0]));
        }
      }
    }
    // ---- the waves' sums together, relative to 2^(r c): 2 and 3 to 0 and 1, 1 to 0
    st.l = sum16x32(st.l) * __builtin_amdgcn_exp2f(-st.k);
    if (g == 0) {
      rst[wave][n][0] = st.r;
      rst[wave][n][1] = st.l;
    }
    lds_barrier();
    float r = rst[0][n][0];
#pragma unroll
    for (int w = 1; w < kAttendWaves; ++w) r = fmaxf(r, rst[w][n][0]);
    float l = 0.f;
#pragma unroll
    for (int w = 0; w < kAttendWaves; ++w)
      l += rst[w][n][1] * __builtin_amdgcn_exp2f((rst[w][n][0] - r) * a.c);
    const float f = __builtin_amdgcn_exp2f(__builtin_fmaf(st.r - r, a.c, -st.k));
    // a lane's 16 dims of a group: 4 i + j
    auto put = [&](float* to) {
#pragma unroll
      for (int c = 0; c < G; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          *(f32x4*)(to + n * kRow + c * 64 + g * 16 + 4 * i) =
              f32x4{st.o[c][0][i], st.o[c][1][i], st.o[c][2][i], st.o[c][3][i]};
    };
    auto add = [&](const float* from) {
#pragma unroll
      for (int c = 0; c < G; ++c)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const f32x4 v = *(const f32x4*)(from + n * kRow + c * 64 + g * 16 + 4 * i);
#pragma unroll
          for (int j = 0; j < 4; ++j) st.o[c][j][i] += v[j];
        }
    };
#pragma unroll
    for (int c = 0; c < G; ++c)
#pragma unroll
      for (int j = 0; j < 4; ++j) st.o[c][j] *= f;
    const int parts = min(last - first, kAttendWaves);       // waves that had tiles
    float* const mine = red + (wave & 1) * kAttendRows * kRow;
    if (wave >= 2 && wave < parts) put(mine);
    lds_barrier();
    if (wave + 2 < parts) add(mine);
    if (wave == 1 && wave < parts) put(mine);
    lds_barrier();
    if (wave == 0) {
      if (parts > 1) add(red + kAttendRows * kRow);
      const bool cut_front = pos > tiles0, cut_back = to < begin + units;
      if (n < rows) {
        const int h = head * a.ratio + row0 + n;
        if (cut_front || cut_back) {
          const int64_t slot = (2 * (int64_t)blockIdx.x + (cut_front ? 0 : 1)) * a.rows + n;
#pragma unroll
          for (int c = 0; c < G; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i)
              *(f32x4*)(a.part + slot * D + c * 64 + g * 16 + 4 * i) =
                  f32x4{st.o[c][0][i], st.o[c][1][i], st.o[c][2][i], st.o[c][3][i]};
          if (g == 0) {
            a.stat[slot * 2] = r;
            a.stat[slot * 2 + 1] = l;
          }
        } else {
          const float inv = l == 0.f ? 0.f : 1.f / l;
          const int64_t out = b * a.ldo + (int64_t)h * D + g * 16;
#pragma unroll
          for (int c = 0; c < G; ++c)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const f32x4 v{st.o[c][0][i] * inv, st.o[c][1][i] * inv, st.o[c][2][i] * inv,
                            st.o[c][3][i] * inv};
              if (a.o != nullptr) *(f32x4*)(a.o + out + c * 64 + 4 * i) = v;
              if (a.o16 != nullptr) {
                typedef f16 f16x4 __attribute__((ext_vector_type(4)));
                *(f16x4*)(a.o16 + out + c * 64 + 4 * i) =
                    f16x4{(f16)v[0], (f16)v[1], (f16)v[2], (f16)v[3]};
              }
            }
          if (a.lse != nullptr && g == 0)
            a.lse[(int64_t)b * a.heads + h] =
                l == 0.f ? -__builtin_inff()
                         : __builtin_fmaf(r, a.c, __builtin_log2f(l)) * 0.69314718055994531f;
        }
      }
    }
    lds_barrier();                       // (the next segment writes red and rst again)
    pos = begin + units;
    if (pos >= to) break;
    begin = pos;
    if (++hg == hgs) {
      hg = 0;
      do { units = seen_units(a, ++b); } while (units == 0);
    }
  }
}

// The parts of the sequences that more than one work-group dealt with, and rows without
// tokens: O = sum of 2^((r_i - max) c) O_i over the same of l_i.  One work-group per (sequence, query
// head): a thread per part for its weight, then D / 4 threads per part, 1024 / D of them at
// a time, eight loads of a thread in flight.  Bound by two rounds of loads, one behind the other:
// 4.0 to 5.5 us, of 1 to 1024 parts.
template <int D>
__global__ __launch_bounds__(256) void k_attend_join(const AttendArgs a) {
  constexpr int kLanes = D / 4, kSubs = 256 / kLanes;
  __shared__ float weight[kMaxParts];
  __shared__ f32x4 red[kSubs][kLanes];
  __shared__ float tops[4], sums[4];
  const int lane = lane_id(), wave = wave_id(), tid = threadIdx.x;
  const int b = blockIdx.x, h = blockIdx.y;
  const int hgs = a.kv_heads * a.rts;
  const int kvh = h / a.ratio, r16 = h % a.ratio;
  const int hg = kvh * a.rts + r16 / kAttendRows, r = r16 % kAttendRows;
  int64_t before = 0, all = 0;
  int units = 0;
  for (int base = 0; base < a.s.seqs; base += 64) {
    const int t = base + lane < a.s.seqs ? seen_units(a, base + lane) : 0;
    const int sum = scan64(t);
    if (b >= base && b < base + 64) {
      units = __builtin_amdgcn_readlane(t, b - base);
      before = all + __builtin_amdgcn_readlane(sum, b - base) - units;
    }
    all += __builtin_amdgcn_readlane(sum, 63);
  }
  f32x4 o{};
  float l = 0.f, top = kNoScore;
  const int sub = tid / kLanes, d = tid % kLanes;
  if (units > 0) {
    const int64_t share = unit_share(all * hgs, a.groups);
    const int64_t begin = before * hgs + (int64_t)hg * units, end = begin + units;
    const int64_t w0 = (begin + kStartUnits) / share, w1 = (end - 1) / share;
    if (w0 == w1) return;                // one work-group had all of it
    const int parts = (int)(w1 - w0) + 1;
    // (the first work-group's range begins before or with the tiles: its second place)
    auto place = [&](int i) { return (2 * (w0 + i) + (i == 0)) * a.rows + r; };
    float pm[kMaxParts / 256], pl[kMaxParts / 256];
#pragma unroll
    for (int j = 0; j < kMaxParts / 256; ++j) {
      const int i = j * 256 + tid;
      pm[j] = i < parts ? a.stat[place(i) * 2] : kNoScore;
      pl[j] = i < parts ? a.stat[place(i) * 2 + 1] : 0.f;
      top = fmaxf(top, pm[j]);
    }
    for (int k = 32; k > 0; k /= 2) top = fmaxf(top, __shfl_xor(top, k));
    if (lane == 0) tops[wave] = top;
    __syncthreads();
    for (int w = 0; w < 4; ++w) top = fmaxf(top, tops[w]);
#pragma unroll
    for (int j = 0; j < kMaxParts / 256; ++j) {
      const int i = j * 256 + tid;
      const float f = __builtin_amdgcn_exp2f((pm[j] - top) * a.c);
      if (i < parts) weight[i] = f;
      l += pl[j] * f;
    }
    for (int k = 32; k > 0; k /= 2) l += __shfl_xor(l, k);
    if (lane == 0) sums[wave] = l;
    __syncthreads();
    l = sums[0] + sums[1] + sums[2] + sums[3];
    int i = sub;
    for (; i + 7 * kSubs < parts; i += 8 * kSubs) {
      f32x4 v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j) v[j] = *(const f32x4*)(a.part + place(i + j * kSubs) * D + d * 4);
#pragma unroll
      for (int j = 0; j < 8; ++j) o += v[j] * weight[i + j * kSubs];
    }
    for (; i < parts; i += kSubs) o += *(const f32x4*)(a.part + place(i) * D + d * 4) * weight[i];
    red[sub][d] = o;
    __syncthreads();
  }
  if (sub != 0) return;
  if (units > 0)
    for (int i = 1; i < kSubs; ++i) o += red[i][d];
  o *= l == 0.f ? 0.f : 1.f / l;
  const int64_t out = b * a.ldo + (int64_t)h * D + d * 4;
  if (a.o != nullptr) *(f32x4*)(a.o + out) = o;
  if (a.o16 != nullptr) {
    typedef f16 f16x4 __attribute__((ext_vector_type(4)));
    *(f16x4*)(a.o16 + out) = f16x4{(f16)o[0], (f16)o[1], (f16)o[2], (f16)o[3]};
  }
  if (a.lse != nullptr && d == 0)
    a.lse[(int64_t)b * a.heads + h] =
        l == 0.f ? -__builtin_inff()
                 : __builtin_fmaf(top, a.c, __builtin_log2f(l)) * 0.69314718055994531f;
}

}  // namespace qlin
