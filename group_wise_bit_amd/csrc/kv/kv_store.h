// Quantizing tokens into the cache, and reading them back (gfx950, wave64).
//
// Both are copies with a change of form: their floor is the bytes of the rows and of the
// codes.  A wave takes a part of a tile whose codes are its own whole words in the layout: half of the
// tokens of the keys, a group of 64 dims of the values.  Whole prompts (8 of 2048 tokens, 8 heads of
// 128, keys of 8 bits, values of 4: 94 MB) are written in 26 us (3.6 TB/s) and read back in 17.5
// (5.3 TB/s, a large copy's rate); 16 prompts of up to 4096 tokens of 8 bits (162 MB) are read
// back in 36 us (4.5 TB/s).  (One wave for all parts of a tile and head: slower, its loads wait
// for each other.)  A few tokens take 5 us, a launch and three rounds of dependent loads: offsets
// and lengths, the page, the rows.
#pragma once

#include "kv_layout.h"

#include <type_traits>

namespace qlin {

struct KvStoreArgs {
  KvSeqs s;
  uint8_t* data;
  const f16* x[2];         // keys, values [m, ldx]
  int64_t ldx[2];
  int64_t head_bytes;      // bytes of a page of one head
  int kv_heads;
};

struct KvReadArgs {
  KvSeqs s;
  const uint8_t* data;
  void* x[2];
  int64_t ldx[2];
  int64_t head_bytes;
  int kv_heads;
};

// The tile that a work-group deals with: tile `tile` (floor of position / 32, below 0
// for rows before a sequence's begin) of sequence b, whose rows are row0 + position for
// positions first .. end - 1.
struct KvSpan {
  int b;
  int64_t tile, first, end, row0;
};

// Rows of sequence b, within 0 .. m whatever the offsets hold.
__device__ __forceinline__ void seq_rows(const KvSeqs& s, int b, int& r0, int& r1) {
  if (s.starts == nullptr) {
    r0 = b;
    r1 = b + 1;
  } else {
    r0 = min(max(s.starts[b], 0), s.m);
    r1 = min(max(s.starts[b + 1], r0), s.m);
  }
}

__device__ __forceinline__ int64_t floor32(int64_t p) { return p >> 5; }

// Item `item` of all sequences' tiles, one after the other: each wave adds up the
// tiles of 64 sequences at a time.
__device__ __forceinline__ bool kv_span(const KvSeqs& s, int item, KvSpan& sp) {
  const int lane = lane_id();
  int b = item, rest = 0;
  if (s.starts != nullptr) {
    int before = 0;
    b = -1;
    for (int base = 0; base < s.seqs; base += 64) {
      int n = 0;
      if (base + lane < s.seqs) {
        int r0, r1;
        seq_rows(s, base + lane, r0, r1);
        if (r1 > r0) {
          const int64_t len = s.lengths[base + lane];
          n = (int)(floor32(len - 1) - floor32(len - (r1 - r0)) + 1);
        }
      }
      const int sum = scan64(n);
      const uint64_t past = __ballot(before + sum > item);
      if (past != 0) {
        const int at = __builtin_ctzll(past);
        b = base + at;
        rest = item - before - (__builtin_amdgcn_readlane(sum, at) - __builtin_amdgcn_readlane(n, at));
        break;
      }
      before += __builtin_amdgcn_readlane(sum, 63);
    }
  }
  if (b < 0 || b >= s.seqs) return false;
  int r0, r1;
  seq_rows(s, b, r0, r1);
  const int64_t len = s.lengths[b], p0 = len - (r1 - r0);
  sp.b = b;
  sp.tile = floor32(p0) + rest;
  sp.first = max(p0, sp.tile * kKvTile);
  sp.end = min(len, (sp.tile + 1) * kKvTile);
  sp.row0 = r0 - p0;
  return sp.first < sp.end;
}

// The page of a tile, -1 if its tokens are not there.
__device__ __forceinline__ int kv_page(const KvSeqs& s, const KvSpan& sp) {
  const int64_t p = sp.tile >> s.page_log;
  if (sp.tile < 0 || p >= s.width) return -1;
  const int page = s.table[sp.b * s.ld + p];
  return page >= 0 && page < s.pages ? page : -1;
}

// Rounding takes most of its time in vector instructions (prompts: 36 us before these forms, 26 with
// them, 16 of those issue at 2.4 GHz; the rest is that a wave loads, rounds and stores once, one
// after the other: it waits half of its cycles):
// ranges are taken on packed fp16 pairs, ties looked for in pairs, codes packed by the conversion
// itself, and for values one lane forms the rounding of a token for the 16 that share it.
//
// The range of a group: two fp16 numbers min(w, 0) and min(-w, 0) over its values, the first
// -inf if one of them is not finite.  (v_pk_min_f16 of two numbers; of a NaN the other one.)
constexpr uint32_t kBadRange = 0x0000FC00u;
__device__ __forceinline__ uint32_t pk_min(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("v_pk_min_f16 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}
template <int N>
__device__ __forceinline__ uint32_t range_of(const uint32_t (&w)[N]) {
  typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
  uint32_t lo = 0, hi = 0;
  u16x2 size{};
#pragma unroll
  for (int i = 0; i < N; ++i) {
    lo = pk_min(lo, w[i]);
    hi = pk_max(hi, w[i]);
    const uint32_t m = w[i] & 0x7FFF7FFFu;
    size = __builtin_elementwise_max(size, __builtin_bit_cast(u16x2, m));
  }
  const uint32_t nhi = hi ^ 0x80008000u;
  // (lo, -hi) of the even values, of the odd ones
  const uint32_t r = pk_min(__builtin_amdgcn_perm(nhi, lo, 0x05040100u),
                            __builtin_amdgcn_perm(nhi, lo, 0x07060302u));
  return max((int)size[0], (int)size[1]) >= 0x7C00 ? kBadRange : r;
}
template <int CTRL>
__device__ __forceinline__ uint32_t mov_dpp(uint32_t v) {
  return (uint32_t)__builtin_amdgcn_mov_dpp((int)v, CTRL, 0xF, 0xF, true);
}
// v[t] of eight numbers t over the 16 lanes of a row, in the lanes y % 8 = t: halves of the
// numbers are exchanged between lanes 4, 2 and 1 apart, so that each step halves them.
__device__ __forceinline__ uint32_t row_min_of_8(const uint32_t (&v)[8], int y) {
  uint32_t a[4], b[2];
#pragma unroll
  for (int i = 0; i < 4; ++i) {                // bit 2 of the number, with the lane 4 apart
    const uint32_t keep = y & 4 ? v[4 + i] : v[i], give = y & 4 ? v[i] : v[4 + i];
    a[i] = pk_min(keep, (uint32_t)__builtin_amdgcn_ds_swizzle((int)give, 0x101F));
  }
#pragma unroll
  for (int i = 0; i < 2; ++i) {                // bit 1, with the lane 2 apart
    const uint32_t keep = y & 2 ? a[2 + i] : a[i], give = y & 2 ? a[i] : a[2 + i];
    b[i] = pk_min(keep, mov_dpp<0x4E>(give));
  }
  const uint32_t keep = y & 1 ? b[1] : b[0], give = y & 1 ? b[0] : b[1];
  const uint32_t c = pk_min(keep, mov_dpp<0xB1>(give));
  return pk_min(c, mov_dpp<0x128>(c));         // the other eight lanes (rotated by 8)
}
// A number of lane T of the row.
template <int T>
__device__ __forceinline__ float from_lane(float v) {
  return __builtin_bit_cast(float, mov_dpp<0x150 + T>(__builtin_bit_cast(uint32_t, v)));
}
// The least over the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ uint32_t quarter_min(uint32_t v) {
  const auto a = __builtin_amdgcn_permlane32_swap(v, v, false, false);
  v = pk_min((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(v, v, false, false);
  return pk_min((uint32_t)b[0], (uint32_t)b[1]);
}

// A group's rounding from its range.
struct KvGroup {
  RtnParams p;
  uint16_t scale;
  float zero;
};
// Quotients correctly rounded by one step from y = 1 / b (Markstein): q = a y, r = a - b q
// exactly, q + r y is a / b rounded if y is 1 / b rounded; and 1 / b itself from a y within
// one unit of it, for a b whose fraction is not all ones (15, 255, an fp16 number).
template <int BITS>
__device__ __forceinline__ KvGroup kv_group(uint32_t range) {
  constexpr int qmax = (1 << BITS) - 1;
  const float lo = (float)as_h2(range)[0], nhi = (float)as_h2(range)[1];
  KvGroup g;
  const bool bad = lo < -65504.f;
  constexpr float y = 1.f / qmax;
  const float d = -nhi - lo, q0 = d * y;
  const f16 s16 = (f16)__builtin_fmaf(__builtin_fmaf(-q0, (float)qmax, d), y, q0);
  const float s = bad ? 0.f : (float)s16;
  g.scale = bad ? (uint16_t)0x7E00 : __builtin_bit_cast(uint16_t, s16);
  const float r0 = __builtin_amdgcn_rcpf(s);
  const float r = __builtin_fmaf(__builtin_fmaf(-s, r0, 1.f), r0, r0);
  const bool none = s == 0.f;
  g.p.s = s;
  g.p.r = none ? 0.f : r;
  g.p.hs = none ? -1.f : 0.5f * s;
  // (the quotient of two fp16 numbers, as a value's: -lo is one of them)
  const float z = none ? 0.f : rtn_fix(-lo, __builtin_rintf(-lo * g.p.r), g.p);
  g.zero = clampf(z, 0.f, (float)qmax);
  g.p.lo = -g.zero;
  g.p.hi = none ? 0.f : (float)qmax - g.zero;
  return g;
}
// Values of a pair rounded, with whether one of them is a tie (rtn_fix is then due).
__device__ __forceinline__ bool kv_round(uint32_t pair, const KvGroup& g, float (&q)[2]) {
  bool tie = false;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    bool t;
    q[i] = rtn_raw((float)as_h2(pair)[i], g.p, t);
    tie |= t;
  }
  return tie;
}
__device__ __forceinline__ void kv_fix(uint32_t pair, const KvGroup& g, float (&q)[2]) {
#pragma unroll
  for (int i = 0; i < 2; ++i) q[i] = rtn_fix((float)as_h2(pair)[i], q[i], g.p);
}
// The code of a rounded value, into byte B of `to`.
template <int B>
__device__ __forceinline__ uint32_t kv_byte(float q, const KvGroup& g, uint32_t to) {
  return __builtin_amdgcn_cvt_pk_u8_f32(clampf(q, g.p.lo, g.p.hi) + g.zero, B, to);
}

// One wave per (tile, head, keys or values), and per half tile of keys / group of
// values: a lane takes the codes that are its own in the layout, finds the group's
// range with the lanes that share it, and has whole words.  Tokens of the
// tile that are not written keep theirs: codes of keys go out by the 16 of a
// token, codes of values by half-words, unless the whole tile is written.
template <int D, int BITS, bool VALUES>
__device__ __forceinline__ void kv_store_tile(const KvStoreArgs& a, const KvSpan& sp, uint8_t* tile,
                                              int head, int part, uint8_t* codes, uint16_t* scales,
                                              uint8_t* zeros) {
  constexpr int G = D / 64;
  const int lane = lane_id();
  const int64_t p0 = sp.tile * kKvTile;
  const bool whole = sp.end - sp.first == kKvTile;
  if constexpr (!VALUES) {
    const int g = lane >> 4, r = lane & 15, h = part;
    const int64_t p = p0 + 16 * h + r;
    const bool mine = p >= sp.first && p < sp.end;
    const f16* src = a.x[0] + (sp.row0 + p) * a.ldx[0] + head * D + 16 * g;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      f16x8 w[2] = {};
      if (mine) {
        w[0] = *(const f16x8*)(src + 64 * c);
        w[1] = *(const f16x8*)(src + 64 * c + 8);
      }
      constexpr int words = BITS / 2;          // of 16 codes
      uint32_t out[words], pair[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const u32x4 four = __builtin_bit_cast(u32x4, w[i / 4]);
        pair[i] = four[i % 4];
      }
      if constexpr (BITS == 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = pair[i];
      } else {
        const KvGroup q = kv_group<BITS>(quarter_min(range_of(pair)));
        float v[8][2];
        bool tie = false;
#pragma unroll
        for (int i = 0; i < 8; ++i) tie |= kv_round(pair[i], q, v[i]);
        if (__ballot(tie) != 0) {
#pragma unroll
          for (int i = 0; i < 8; ++i) kv_fix(pair[i], q, v[i]);
        }
        // code i of a word at bit 16 (i % 2) + BITS (i / 2)
#pragma unroll
        for (int i = 0; i < words; ++i) {
          constexpr int per = 16 / BITS;       // pairs of a word
          uint32_t even = 0, odd = 0;          // (4 bits) bytes of pairs 0 and 2, of 1 and 3
          even = kv_byte<0>(v[i * per][0], q, even);
          even = kv_byte<2>(v[i * per][1], q, even);
          if constexpr (BITS == 8) {
            even = kv_byte<1>(v[i * per + 1][0], q, even);
            out[i] = kv_byte<3>(v[i * per + 1][1], q, even);
          } else {
            odd = kv_byte<0>(v[i * per + 1][0], q, odd);
            odd = kv_byte<2>(v[i * per + 1][1], q, odd);
            even = kv_byte<1>(v[i * per + 2][0], q, even);
            even = kv_byte<3>(v[i * per + 2][1], q, even);
            odd = kv_byte<1>(v[i * per + 3][0], q, odd);
            odd = kv_byte<3>(v[i * per + 3][1], q, odd);
            out[i] = even | odd << 4;
          }
        }
        if (mine && g == 0) {
          scales[c * 32 + (r >> 2) * 8 + h * 4 + (r & 3)] = q.scale;
          zeros[(r * 2 + h) * G + c] = (uint8_t)q.zero;
        }
      }
      if (mine) {
        const int at = (h * G + c) * words;    // word of the lane's run
        if constexpr (BITS == 4) {
          *(u32x2*)(codes + ((at / 4 * 64 + lane) * 4 + at % 4) * 4) = u32x2{out[0], out[1]};
        } else {
#pragma unroll
          for (int i = 0; i < words / 4; ++i)
            *(u32x4*)(codes + ((at / 4 + i) * 64 + lane) * 16) =
                u32x4{out[4 * i], out[4 * i + 1], out[4 * i + 2], out[4 * i + 3]};
        }
      }
    }
  } else {
    constexpr int n = 16 / BITS;               // codes of a half-word
    const int g = lane >> 4, y = lane & 15, c = part;
    u32x2 w[8];
    bool mine[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {              // tokens 4 g + t of the first half, then the second
      const int64_t p = p0 + (t >> 2) * 16 + 4 * g + (t & 3);
      mine[t] = p >= sp.first && p < sp.end;
      w[t] = u32x2{0, 0};
      if (mine[t]) w[t] = *(const u32x2*)(a.x[1] + (sp.row0 + p) * a.ldx[1] + head * D + c * 64 + 4 * y);
    }
    uint32_t out[4 / n][4];                    // [part of 4 dims][pair of tokens]
    KvGroup own;                               // of token y % 8
    if constexpr (BITS < 16) {
      uint32_t range[8];
#pragma unroll
      for (int t = 0; t < 8; ++t) {
        const uint32_t pair[2] = {w[t][0], w[t][1]};
        range[t] = range_of(pair);
      }
      own = kv_group<BITS>(row_min_of_8(range, y));
      if (y < 8 && (p0 + (y >> 2) * 16 + 4 * g + (y & 3)) >= sp.first &&
          (p0 + (y >> 2) * 16 + 4 * g + (y & 3)) < sp.end) {
        scales[c * 32 + g * 8 + y] = own.scale;
        zeros[(g * G + c) * 8 + y] = (uint8_t)own.zero;
      }
    }
    auto token = [&](auto T) {                 // a token's rounding, from the lane that has it
      constexpr int t = decltype(T)::value;
      KvGroup q;
      q.p.s = from_lane<t>(own.p.s);
      q.p.r = from_lane<t>(own.p.r);
      q.p.hs = from_lane<t>(own.p.hs);
      q.p.hi = from_lane<t>(own.p.hi);
      q.zero = from_lane<t>(own.zero);
      q.p.lo = -q.zero;
      q.scale = 0;
      return q;
    };
    auto two = [&](auto U) {                   // tokens 2 u (low halves) and 2 u + 1
      constexpr int u = decltype(U)::value;
      const uint32_t pair[2][2] = {{w[2 * u][0], w[2 * u][1]}, {w[2 * u + 1][0], w[2 * u + 1][1]}};
      if constexpr (BITS == 16) {
        out[0][u] = __builtin_amdgcn_perm(pair[1][0], pair[0][0], 0x05040100u);
        out[1][u] = __builtin_amdgcn_perm(pair[1][0], pair[0][0], 0x07060302u);
        out[2][u] = __builtin_amdgcn_perm(pair[1][1], pair[0][1], 0x05040100u);
        out[3][u] = __builtin_amdgcn_perm(pair[1][1], pair[0][1], 0x07060302u);
      } else {
        float v[2][2][2];                      // [token][pair][value]
        const KvGroup q[2] = {token(std::integral_constant<int, 2 * u>{}),
                              token(std::integral_constant<int, 2 * u + 1>{})};
        bool tie = false;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int i = 0; i < 2; ++i) tie |= kv_round(pair[k][i], q[k], v[k][i]);
        if (__ballot(tie) != 0) {
#pragma unroll
          for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int i = 0; i < 2; ++i) kv_fix(pair[k][i], q[k], v[k][i]);
        }
        if constexpr (BITS == 8) {
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            uint32_t o = kv_byte<0>(v[0][i][0], q[0], 0);
            o = kv_byte<1>(v[0][i][1], q[0], o);
            o = kv_byte<2>(v[1][i][0], q[1], o);
            out[i][u] = kv_byte<3>(v[1][i][1], q[1], o);
          }
        } else {
          uint32_t even = 0, odd = 0;          // bytes of dims 0 and 2, of 1 and 3
          even = kv_byte<0>(v[0][0][0], q[0], even);
          odd = kv_byte<0>(v[0][0][1], q[0], odd);
          even = kv_byte<1>(v[0][1][0], q[0], even);
          odd = kv_byte<1>(v[0][1][1], q[0], odd);
          even = kv_byte<2>(v[1][0][0], q[1], even);
          odd = kv_byte<2>(v[1][0][1], q[1], odd);
          even = kv_byte<3>(v[1][1][0], q[1], even);
          odd = kv_byte<3>(v[1][1][1], q[1], odd);
          out[0][u] = even | odd << 4;
        }
      }
    };
    two(std::integral_constant<int, 0>{});
    two(std::integral_constant<int, 1>{});
    two(std::integral_constant<int, 2>{});
    two(std::integral_constant<int, 3>{});
    if (whole) {
#pragma unroll
      for (int i = 0; i < 4 / n; ++i)
        *(u32x4*)(codes + ((c * (4 / n) + i) * 64 + lane) * 16) =
            u32x4{out[i][0], out[i][1], out[i][2], out[i][3]};
    } else {
#pragma unroll
      for (int i = 0; i < 4 / n; ++i)
#pragma unroll
        for (int t = 0; t < 8; ++t)
          if (mine[t])
            *(uint16_t*)(codes + ((c * (4 / n) + i) * 64 + lane) * 16 + t * 2) =
                (uint16_t)(out[i][t / 2] >> (16 * (t % 2)));
    }
  }
}

// Waves of a tile and head: 2 for the halves of the keys, G for the groups of values.
template <int D, int KB, int VB>
__global__ __launch_bounds__(256) void k_kv_store(const KvStoreArgs a) {
  using T = KvTile<D, KB, VB>;
  KvSpan sp;
  if (!kv_span(a.s, blockIdx.x, sp)) return;
  const int part = blockIdx.y * 4 + wave_id();
  const int head = part / (2 + T::G), which = part % (2 + T::G);
  if (head >= a.kv_heads) return;
  const int page = kv_page(a.s, sp);
  if (page < 0) return;
  uint8_t* tile = a.data + ((int64_t)page * a.kv_heads + head) * a.head_bytes +
                  (sp.tile & ((1 << a.s.page_log) - 1)) * T::bytes;
  if (which < 2)
    kv_store_tile<D, KB, false>(a, sp, tile, head, which, tile + T::k, (uint16_t*)(tile + T::ks),
                                tile + T::kz);
  else
    kv_store_tile<D, VB, true>(a, sp, tile, head, which - 2, tile + T::v, (uint16_t*)(tile + T::vs),
                               tile + T::vz);
}

// ------------------------------------------------------------------ reading
template <bool WIDE, bool KEPT>
__device__ __forceinline__ void put(void* base, int64_t at, const float* v, int count) {
  if constexpr (WIDE) {
    float* o = (float*)base + at;
    for (int i = 0; i < count; i += 4) *(f32x4*)(o + i) = f32x4{v[i], v[i + 1], v[i + 2], v[i + 3]};
  } else {
    typedef f16 f16x4 __attribute__((ext_vector_type(4)));
    f16* o = (f16*)base + at;
    for (int i = 0; i < count; i += 4) {
      f16x4 r;
      for (int j = 0; j < 4; ++j) {
        float x = v[i + j];
        if (!KEPT && __builtin_fabsf(x) > 65504.f) x = __builtin_copysignf(65504.f, x);
        r[j] = (f16)x;
      }
      *(f16x4*)(o + i) = r;
    }
  }
}

// The same split: a lane reads its own words of the layout, and writes 16 dims of a
// token's key, or 4 dims of 8 tokens' values.
template <int D, int BITS, bool VALUES, bool WIDE>
__device__ __forceinline__ void kv_read_tile(const KvReadArgs& a, const KvSpan& sp, bool there,
                                             int head, int part, const uint8_t* codes,
                                             const uint16_t* scales, const uint8_t* zeros) {
  constexpr int G = D / 64;
  const int lane = lane_id();
  const int64_t p0 = sp.tile * kKvTile;
  if constexpr (!VALUES) {
    const int g = lane >> 4, r = lane & 15, h = part;
    const int64_t p = p0 + 16 * h + r;
    if (p < sp.first || p >= sp.end) return;
    constexpr int words = BITS / 2, per = 32 / BITS;
#pragma unroll
    for (int c = 0; c < G; ++c) {
      float v[16] = {};
      if (there) {
        const int at = (h * G + c) * words;
        uint32_t w[words];
        if constexpr (BITS == 4) {
          const u32x2 u = *(const u32x2*)(codes + ((at / 4 * 64 + lane) * 4 + at % 4) * 4);
          w[0] = u[0];
          w[1] = u[1];
        } else {
#pragma unroll
          for (int i = 0; i < words / 4; ++i) {
            const u32x4 u = *(const u32x4*)(codes + ((at / 4 + i) * 64 + lane) * 16);
#pragma unroll
            for (int j = 0; j < 4; ++j) w[4 * i + j] = u[j];
          }
        }
        float s = 1.f;
        int z = 0;
        if constexpr (BITS < 16) {
          s = h2f(scales[c * 32 + (r >> 2) * 8 + h * 4 + (r & 3)]);
          z = zeros[(r * 2 + h) * G + c];
        }
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const int j = i % per;
          const uint32_t code = (w[i / per] >> (16 * (j % 2) + BITS * (j / 2))) & ((1u << BITS) - 1);
          v[i] = BITS == 16 ? h2f((uint16_t)code) : s * (float)((int)code - z);
        }
      }
      put<WIDE, BITS == 16>(a.x[0], (sp.row0 + p) * a.ldx[0] + head * D + c * 64 + 16 * g, v, 16);
    }
  } else {
    constexpr int n = 16 / BITS;
    const int g = lane >> 4, y = lane & 15, c = part;
    u32x4 w[4 / n] = {}, s = {};
    u32x2 z = {};
    if (there) {
#pragma unroll
      for (int i = 0; i < 4 / n; ++i) w[i] = *(const u32x4*)(codes + ((c * (4 / n) + i) * 64 + lane) * 16);
      if constexpr (BITS < 16) {
        s = *(const u32x4*)(scales + c * 32 + g * 8);
        z = *(const u32x2*)(zeros + (g * G + c) * 8);
      }
    }
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      const int64_t p = p0 + (t >> 2) * 16 + 4 * g + (t & 3);
      if (p < sp.first || p >= sp.end) continue;
      const float sc = h2f((uint16_t)(s[t / 2] >> (16 * (t % 2))));
      const int ze = (z[t / 4] >> (8 * (t % 4))) & 255;
      float v[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t code = (w[j / n][t / 2] >> (16 * (t % 2) + BITS * (j % n))) & ((1u << BITS) - 1);
        v[j] = BITS == 16 ? h2f((uint16_t)code) : sc * (float)((int)code - ze);
      }
      put<WIDE, BITS == 16>(a.x[1], (sp.row0 + p) * a.ldx[1] + head * D + c * 64 + 4 * y, v, 4);
    }
  }
}

template <int D, int KB, int VB, bool WIDE>
__global__ __launch_bounds__(256) void k_kv_read(const KvReadArgs a) {
  using T = KvTile<D, KB, VB>;
  KvSpan sp;
  if (!kv_span(a.s, blockIdx.x, sp)) return;
  const int part = blockIdx.y * 4 + wave_id();
  const int head = part / (2 + T::G), which = part % (2 + T::G);
  if (head >= a.kv_heads) return;
  const int page = kv_page(a.s, sp);
  const uint8_t* tile = a.data + ((int64_t)max(page, 0) * a.kv_heads + head) * a.head_bytes +
                        (sp.tile & ((1 << a.s.page_log) - 1)) * T::bytes;
  if (which < 2)
    kv_read_tile<D, KB, false, WIDE>(a, sp, page >= 0, head, which, tile + T::k,
                                     (const uint16_t*)(tile + T::ks), tile + T::kz);
  else
    kv_read_tile<D, VB, true, WIDE>(a, sp, page >= 0, head, which - 2, tile + T::v,
                                    (const uint16_t*)(tile + T::vs), tile + T::vz);
}

}  // namespace qlin
