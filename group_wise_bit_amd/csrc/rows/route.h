// Routing to experts (gfx950, wave64).
#pragma once

#include "../device_common.h"

#include <type_traits>

namespace qlin {

struct RouteArgs {
  const float* logits;
  const float* bias;
  int64_t ld;
  int32_t* ids;
  float* weights;
  int m, experts, top_k, groups, top_groups, group_top;
  float scale;
  bool sigmoid, renormalize;
};

constexpr int kRouteWaves = 4;

// One wave per row, lane l holds experts EPL l .. EPL l + EPL - 1.  The choice
// is that of 64-bit scores.  Without a bias and with groups of one best the keys
// are logits and 32 bits are exact.  Otherwise scores are formed in 32 bits
// first, each key within slack() of its exact value, and the choice stands if
// every two neighbours in it -- and the last one in and the first one out -- are
// further apart than that; a row that cannot be told apart so (2 in 1000 of 256
// random experts) is done again in 64 bits.  Keys are held as integers of the
// same order (0: a masked expert), so that a DPP maximum is one instruction;
// the best one is read into a scalar, and its lane and place are found by scalar
// instructions, the lowest first.  Bound by instruction issue: a row of 256 experts in 8
// groups takes 637 vector and 662 scalar instructions, and in 26.4 us for 16384 of them
// a vector one issues in 77 % of a SIMD's cycles, a scalar one in 76 %; 64 bits
// throughout took 57 us.
template <int CTRL>
__device__ __forceinline__ uint32_t dpp_u(uint32_t v) {   // (lanes that receive nothing: 0)
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, 0xF, 0xF, false);
}
template <int CTRL>
__device__ __forceinline__ uint64_t dpp_u(uint64_t v) {
  return (uint64_t)dpp_u<CTRL>((uint32_t)v) | ((uint64_t)dpp_u<CTRL>((uint32_t)(v >> 32)) << 32);
}
template <int CTRL>
__device__ __forceinline__ float dpp_u(float v) {
  return __builtin_bit_cast(float, dpp_u<CTRL>(__builtin_bit_cast(uint32_t, v)));
}
template <int CTRL>
__device__ __forceinline__ double dpp_u(double v) {
  return __builtin_bit_cast(double, dpp_u<CTRL>(__builtin_bit_cast(uint64_t, v)));
}
__device__ __forceinline__ uint32_t lane_u(uint32_t v, int l) {
  return (uint32_t)__builtin_amdgcn_readlane((int)v, l);
}
__device__ __forceinline__ uint64_t lane_u(uint64_t v, int l) {
  return (uint64_t)lane_u((uint32_t)v, l) | ((uint64_t)lane_u((uint32_t)(v >> 32), l) << 32);
}
// The wave's maximum / sum: within rows of 16 lanes (pairs, quads, mirrors),
// then row 0 into 1 and 2 into 3 (row_bcast15), then rows 0-1 into 2-3
// (row_bcast31); lane 63 has it all.  64 bits: the high halves' maximum, then the
// low halves' of the lanes that have it.
__device__ __forceinline__ uint32_t max64(uint32_t v) {
  v = max(v, dpp_u<0xB1>(v));
  v = max(v, dpp_u<0x4E>(v));
  v = max(v, dpp_u<0x141>(v));
  v = max(v, dpp_u<0x140>(v));
  v = max(v, dpp_u<0x142>(v));
  v = max(v, dpp_u<0x143>(v));
  return lane_u(v, 63);
}
__device__ __forceinline__ uint64_t max64(uint64_t v) {
  const uint32_t hi = max64((uint32_t)(v >> 32));
  return ((uint64_t)hi << 32) | max64((uint32_t)(v >> 32) == hi ? (uint32_t)v : 0u);
}
template <typename T>
__device__ __forceinline__ T sum64(T v) {
  v += dpp_u<0xB1>(v);
  v += dpp_u<0x4E>(v);
  v += dpp_u<0x141>(v);
  v += dpp_u<0x140>(v);
  v += dpp_u<0x142>(v);
  v += dpp_u<0x143>(v);
  if constexpr (sizeof(T) == 4) return __builtin_bit_cast(T, lane_u(__builtin_bit_cast(uint32_t, v), 63));
  else return __builtin_bit_cast(T, lane_u(__builtin_bit_cast(uint64_t, v), 63));
}
// Integers in the order of floats (-0 as +0; every float above -infinity is
// above 0), and back.
__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __builtin_bit_cast(uint32_t, v + 0.f);
  return b ^ ((uint32_t)((int32_t)b >> 31) | 0x80000000u);
}
__device__ __forceinline__ uint64_t ordered(double v) {
  const uint64_t b = __builtin_bit_cast(uint64_t, v + 0.0);
  return b ^ ((uint64_t)((int64_t)b >> 63) | 0x8000000000000000ull);
}
__device__ __forceinline__ float unordered(uint32_t k) {
  return __builtin_bit_cast(float, k ^ ((uint32_t)((int32_t)~k >> 31) | 0x80000000u));
}
__device__ __forceinline__ double unordered(uint64_t k) {
  return __builtin_bit_cast(double, k ^ ((uint64_t)((int64_t)~k >> 63) | 0x8000000000000000ull));
}

// How far a key formed in 32 bits can be from its exact value, with u = 2^-24.
// Sigmoid: the exponential is off by 2u (1 ulp) + 1.5u |x| (its argument's rounding),
// which p (1 - p) <= 1/4, p (1 - p) |x| <= 0.23 times reaches p; the sum's rounding
// and the reciprocal (1 ulp) are 3u: under 4u in all, taken as 6u < 3.6e-7.
// Softmax, d = top - x: the exponential is off by 2u + 2.5u d (the difference's and
// its argument's rounding).  The sum is off by its terms' mean of that, and a mean
// of d over 512 experts or fewer is below 3.9, and by 13u of its additions (7 in a
// lane, 6 across lanes): 25u; the reciprocal and the product are 3u.  With p <= 1 and
// p d <= 0.37 that is under 31u, taken as 40u < 2.4e-6.  And the rounding of the sum
// with the bias, u |key|.
__device__ __forceinline__ float slack(const RouteArgs& a, float key) {
  return (a.sigmoid ? 3.6e-7f : 2.4e-6f) + 6e-8f * __builtin_fabsf(key);
}

// exp(x - top) for finite x <= top, the rounding error of the difference (Knuth's
// two-sum of x and -top) added back: 3 half steps wherever it is normal.
__device__ __forceinline__ float exp_below(float x, float top) {
  const float d = x - top;
  if (d < -110.f) return 0.f;                // (below fp32's smallest number)
  const float b = d - x;
  const float err = (x - (d - b)) + (-top - b);
  return expf(d) * (1.f + err);
}

// One row with scores of type T.  False (nothing written) if 32 bits cannot
// tell the choice.  val: 64 EPL keys of LDS, the wave's own.
template <int EPL, typename T>
__device__ __forceinline__ bool route_row(const RouteArgs& a, int row, void* val) {
  constexpr bool kExact = sizeof(T) == 8;
  using K = typename std::conditional<kExact, uint64_t, uint32_t>::type;
  constexpr float kInf = __builtin_inff();
  constexpr float kMax = 3.402823466e38f;
  const int lane = lane_id();
  const float* lp = a.logits + (int64_t)row * a.ld;
  const int e0 = EPL * lane;
  float x[EPL], bias[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) x[i] = lp[min(e0 + i, a.experts - 1)];
  if (a.bias != nullptr) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) bias[i] = a.bias[min(e0 + i, a.experts - 1)];
  }
  // logits, +inf as the largest finite one; live: not masked (-inf, NaN)
  bool live[EPL];
  K key[EPL];
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    live[i] = e0 + i < a.experts && x[i] > -kInf;
    x[i] = __builtin_fminf(x[i], kMax);
    key[i] = live[i] ? ordered((T)x[i]) : 0;
    most = max(most, live[i] ? ordered(x[i]) : 0u);
  }
  const bool scored = a.bias != nullptr || (a.groups > 1 && a.group_top == 2);
  float top = 0.f;
  T total = 1;                               // of the softmax
  T p[EPL];
  if (!a.sigmoid) {
    most = max64(most);
    top = most != 0 ? unordered(most) : 0.f;
    if (scored || !a.renormalize) {
      total = 0;
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        if constexpr (kExact) p[i] = live[i] ? exp((T)x[i] - (T)top) : 0;
        else p[i] = live[i] ? __expf(x[i] - top) : 0;
        total += p[i];
      }
      total = sum64(total);
      if (total > 0) {
#pragma unroll
        for (int i = 0; i < EPL; ++i) {
          if constexpr (kExact) p[i] /= total;
          else p[i] *= __builtin_amdgcn_rcpf(total);
        }
      }
    }
  } else if (scored) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if constexpr (kExact) p[i] = 1 / (1 + exp(-(T)x[i]));
      else p[i] = __builtin_amdgcn_rcpf(1.f + __expf(-x[i]));
    }
  }
  if (a.bias != nullptr) {
    // (a bias of -inf or NaN masks the expert)
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      key[i] = live[i] && bias[i] > -kInf ? ordered(p[i] + (T)bias[i]) : 0;
  }
  // whether 32 bits leave it open which of two keys is larger
  auto close = [&](K larger, K smaller) __attribute__((always_inline)) {
    if constexpr (kExact) return false;
    const float v = unordered((uint32_t)larger);
    return !(v - unordered((uint32_t)smaller) > 2.f * slack(a, v));
  };
  if (a.groups > 1) {
    const int per = a.experts / a.groups;
    K* v = static_cast<K*>(val);
    // (two scores: without a bias the scores' own order is the keys')
    const bool scores = a.group_top == 2 && a.bias == nullptr;
#pragma unroll
    for (int i = 0; i < EPL; ++i) v[e0 + i] = scores && key[i] != 0 ? ordered(p[i]) : key[i];
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    // 2^s lanes per group, each the two best of every 2^s-th member, then of all
    const int s = __builtin_clz(a.groups - 1) - 26;        // 64 >> ceil(log2(groups)) lanes
    const int g = lane >> s, n = 1 << s;
    K first = 0, second = 0;
    if (g < a.groups)
      for (int j = lane & (n - 1); j < per; j += n) {
        const K w = v[g * per + j];
        second = max(second, min(first, w));
        first = max(first, w);
      }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    auto merge = [&](K f, K w) __attribute__((always_inline)) {
      second = max(min(first, f), max(second, w));
      first = max(first, f);
    };
    if (s > 0) merge(dpp_u<0xB1>(first), dpp_u<0xB1>(second));
    if (s > 1) merge(dpp_u<0x4E>(first), dpp_u<0x4E>(second));
    if (s > 2) merge(dpp_u<0x141>(first), dpp_u<0x141>(second));
    if (s > 3) merge(dpp_u<0x140>(first), dpp_u<0x140>(second));
    if (s > 4) merge(__shfl_xor(first, 16), __shfl_xor(second, 16));
    const K value =
        a.group_top == 1 || second == 0 ? first : ordered(unordered(first) + unordered(second));
    K gv = value;
    uint64_t kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      const K best = max64(gv);
      if (best == 0) break;
      const int at = __builtin_ctzll(__builtin_amdgcn_ballot_w64(gv == best)) >> s;
      kept |= 1ull << at;
      gv = g == at ? 0 : gv;
    }
    // 32 bits tell the groups apart if the least that a kept one can be is above the
    // most that one left out can be.  A value is off by its scores' errors and the
    // rounding of their sum (6e-8 of their sizes, not of the sum's: they may cancel),
    // and as much again is taken for the bound's own rounding.
    if constexpr (!kExact) {
      if (scored) {
        const float v = unordered(value), v1 = unordered(first);
        const bool two = a.group_top == 2 && second != 0;
        const float v2 = two ? unordered(second) : 0.f;
        const float off = slack(a, v1) + (two ? slack(a, v2) : 0.f) + 1.2e-7f * __builtin_fabsf(v1) +
                          1.2e-7f * __builtin_fabsf(v2);
        const bool in = (kept >> g) & 1;
        float x = in ? off - v : off + v;
        x = x < kInf ? x : kInf;             // (NaN: it cannot be told)
        const uint32_t least = max64(in && value != 0 ? ordered(x) : 0u);
        const uint32_t most_out = max64(!in && value != 0 ? ordered(x) : 0u);
        if (least != 0 && most_out != 0 && !(unordered(least) + unordered(most_out) < 0.f)) return false;
      }
    }
    const float inv = 1.f / (float)per;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      // the group of expert e: (e + 1/2) / per is at least 1/1024 from an integer
      const int ge = (int)(((float)(e0 + i) + 0.5f) * inv);
      if (!((kept >> (ge & 63)) & 1)) key[i] = 0;
    }
  }
  // the best top_k; lane j keeps the j-th
  int mine = -1;
  K last = 0;
  for (int j = 0; j <= a.top_k; ++j) {
    if (j == a.top_k && (kExact || a.bias == nullptr)) break;
    K mx = key[0];
#pragma unroll
    for (int i = 1; i < EPL; ++i) mx = max(mx, key[i]);
    const K best = max64(mx);
    if (best == 0) break;
    if (a.bias != nullptr && j > 0 && close(last, best)) return false;
    if (j == a.top_k) break;
    last = best;
    // the lowest expert that has it: the first lane, and its first place
    const int l = __builtin_ctzll(__builtin_amdgcn_ballot_w64(mx == best));
    int place = EPL - 1;
#pragma unroll
    for (int i = EPL - 2; i >= 0; --i) place = lane_u(key[i], l) == best ? i : place;
#pragma unroll
    for (int i = 0; i < EPL; ++i) key[i] = lane == (place == i ? l : -1) ? 0 : key[i];
    mine = lane == j ? EPL * l + place : mine;
  }
  // the chosen ones' scores
  float xm = 0.f;
  T w = 0;
  if (mine >= 0) xm = __builtin_fminf(lp[mine], kMax);
  if constexpr (kExact) {
    if (mine >= 0) w = a.sigmoid ? 1 / (1 + exp(-(T)xm)) : exp((T)xm - (T)top);
  } else {
    // (a score this small, exp(-80) = 1.8e-35 of a softmax's largest, is left to 64 bits:
    // fp32 has few or no bits of it, and renormalizing or the scale can make it large.
    // With a bias all of the chosen can be so far below the row's largest logit.)
    const float below = a.sigmoid ? xm : xm - top;
    if (__builtin_amdgcn_ballot_w64(mine >= 0 && below < -80.f) != 0) return false;
    if (mine >= 0) w = a.sigmoid ? 1.f / (1.f + expf(-xm)) : exp_below(xm, top);
  }
  const T sum = a.renormalize ? sum64(w) : total;
  if (lane < a.top_k) {
    const int64_t o = (int64_t)row * a.top_k + lane;
    a.ids[o] = mine;
    a.weights[o] = sum > 0 ? (float)(w / sum * (T)a.scale) : 0.f;
  }
  return true;
}

template <int EPL>
__global__ __launch_bounds__(kRouteWaves * 64) void k_route(const RouteArgs a) {
  __shared__ uint64_t val[kRouteWaves][EPL * 64];
  const int wave = wave_id(), row = blockIdx.x * kRouteWaves + wave;
  if (row >= a.m) return;
  if (!route_row<EPL, float>(a, row, val[wave])) route_row<EPL, double>(a, row, val[wave]);
}

}  // namespace qlin
