// Quantizing tokens into the cache, and reading them back (gfx950, wave64).
#pragma once

#include "kv_layout.h"

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

template <int CTRL>
__device__ __forceinline__ float mov_dpp(float v) {
  return __builtin_bit_cast(float, __builtin_amdgcn_mov_dpp(__builtin_bit_cast(int, v), CTRL, 0xF,
                                                            0xF, true));
}
// Minimum over the 16 lanes of a row (pairs, quads, mirrors of 8 and 16), and over
// the four lanes l, l ^ 16, l ^ 32, l ^ 48.
__device__ __forceinline__ float row_min(float v) {
  v = fminf(v, mov_dpp<0xB1>(v));
  v = fminf(v, mov_dpp<0x4E>(v));
  v = fminf(v, mov_dpp<0x141>(v));
  return fminf(v, mov_dpp<0x140>(v));
}
__device__ __forceinline__ float quarter_min(float v) {
  v = fminf(v, __shfl_xor(v, 16));
  return fminf(v, __shfl_xor(v, 32));
}

// A group's rounding from lo = min(w, 0), or -inf for a group that is not finite, and nhi =
// -max(w, 0).
struct KvGroup {
  RtnParams p;
  uint16_t scale;
  int zero;
};
template <int BITS>
__device__ __forceinline__ KvGroup kv_group(float lo, float nhi) {
  constexpr int qmax = (1 << BITS) - 1;
  KvGroup g;
  if (lo < -65504.f) {
    g.p = rtn_params(0.f, 0, qmax);
    g.scale = 0x7E00;
    g.zero = 0;
    return g;
  }
  const f16 s = (f16)__fdiv_rn(-nhi - lo, (float)qmax);
  g.scale = __builtin_bit_cast(uint16_t, s);
  g.zero = 0;
  g.p = rtn_params((float)s, 0, qmax);
  if ((float)s != 0.f) {
    // (the quotient of two fp16 numbers, as a weight's: -lo is one of the values)
    const float z = rtn_fix(-lo, __builtin_rintf(-lo * g.p.r), g.p);
    g.zero = (int)clampf(z, 0.f, (float)qmax);
    g.p = rtn_params((float)s, g.zero, qmax);
  }
  return g;
}
__device__ __forceinline__ uint32_t kv_code(f16 w, const KvGroup& g) {
  if (g.p.s == 0.f) return 0;
  const float q = rtn_fix((float)w, __builtin_rintf((float)w * g.p.r), g.p);
  return (uint32_t)((int)clampf(q, g.p.lo, g.p.hi) + g.zero);
}

// One value's part in its group's (lo, nhi): a value that is not finite makes lo -inf.
__device__ __forceinline__ void kv_range(f16 w, float& lo, float& nhi) {
  const float x = (float)w;
  const bool ok = __builtin_fabsf(x) <= 65504.f;
  lo = ok ? fminf(lo, x) : -__builtin_inff();
  nhi = ok ? fminf(nhi, -x) : nhi;
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
      uint32_t out[words];
      if constexpr (BITS == 16) {
#pragma unroll
        for (int i = 0; i < 8; ++i) out[i] = __builtin_bit_cast(u32x4, w[i / 4])[i % 4];
      } else {
        float lo = 0.f, nhi = 0.f;
#pragma unroll
        for (int i = 0; i < 16; ++i) kv_range(w[i / 8][i % 8], lo, nhi);
        const KvGroup q = kv_group<BITS>(quarter_min(lo), quarter_min(nhi));
        constexpr int per = 32 / BITS;
#pragma unroll
        for (int i = 0; i < words; ++i) {
          out[i] = 0;
#pragma unroll
          for (int j = 0; j < per; ++j) {
            const int e = i * per + j;
            out[i] |= kv_code(w[e / 8][e % 8], q) << (16 * (j % 2) + BITS * (j / 2));
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
    typedef f16 f16x4 __attribute__((ext_vector_type(4)));
    constexpr int n = 16 / BITS;               // codes of a half-word
    const int g = lane >> 4, y = lane & 15, c = part;
    f16x4 w[8];
    bool mine[8];
#pragma unroll
    for (int t = 0; t < 8; ++t) {              // tokens 4 g + t of the first half, then the second
      const int64_t p = p0 + (t >> 2) * 16 + 4 * g + (t & 3);
      mine[t] = p >= sp.first && p < sp.end;
      w[t] = f16x4{};
      if (mine[t]) w[t] = *(const f16x4*)(a.x[1] + (sp.row0 + p) * a.ldx[1] + head * D + c * 64 + 4 * y);
    }
    uint32_t out[4 / n][4] = {};               // [part of 4 dims][pair of tokens]
#pragma unroll
    for (int t = 0; t < 8; ++t) {
      uint32_t code[4];
      if constexpr (BITS == 16) {
#pragma unroll
        for (int j = 0; j < 4; ++j) code[j] = __builtin_bit_cast(uint16_t, (f16)w[t][j]);
      } else {
        float lo = 0.f, nhi = 0.f;
#pragma unroll
        for (int j = 0; j < 4; ++j) kv_range(w[t][j], lo, nhi);
        const KvGroup q = kv_group<BITS>(row_min(lo), row_min(nhi));
#pragma unroll
        for (int j = 0; j < 4; ++j) code[j] = kv_code(w[t][j], q);
        if (mine[t] && y == 0) {
          scales[c * 32 + g * 8 + t] = q.scale;
          zeros[(g * G + c) * 8 + t] = (uint8_t)q.zero;
        }
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) out[j / n][t / 2] |= code[j] << (16 * (t % 2) + BITS * (j % n));
    }
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
