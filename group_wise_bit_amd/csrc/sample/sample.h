// Drawing a token from a row of logits (gfx950, wave64).
#pragma once

#include "../device_common.h"

#include <float.h>

namespace qlin {

struct SampleArgs {
  const float* temperature;
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const float* logits;
  const float* u;
  int64_t ld;
  int32_t* ids;
  float* probs;
  int m, vocab;
};

// A row's settings, with what is off or out of range put in order.
struct SampleRow {
  double t;          // temperature; 0: the first of the largest logits is taken
  int k;             // 0: off
  float p, mp, u;    // p 1, mp 0: off
};

// (every load is made, of u where a setting is off, so that they are in flight together)
__device__ __forceinline__ SampleRow sample_row(const SampleArgs& a, int row) {
  const float u = a.u[row];
  const float tv = (a.temperature != nullptr ? a.temperature : a.u)[row];
  const int kv = (a.top_k != nullptr ? a.top_k : reinterpret_cast<const int32_t*>(a.u))[row];
  const float pv = (a.top_p != nullptr ? a.top_p : a.u)[row];
  const float mv = (a.min_p != nullptr ? a.min_p : a.u)[row];
  const float t = a.temperature != nullptr ? tv : 1.f;
  const int k = a.top_k != nullptr ? kv : 0;
  const float p = a.top_p != nullptr ? pv : 1.f;
  const float mp = a.min_p != nullptr ? mv : 0.f;
  SampleRow r;
  // (with min_p above 1 no p reaches it: the first token alone, as with top_k 1)
  r.t = t > 0.f && k != 1 && !(mp > 1.f) ? (double)t : 0.;
  r.k = k > 0 && k < a.vocab ? k : 0;
  r.p = p < 1.f ? fmaxf(p, 0.f) : 1.f;
  r.mp = mp > 0.f ? mp : 0.f;
  r.u = u > 0.f ? u : 0.f;
  return r;
}

// A logit as it counts: +inf is the largest finite number, -inf and NaN (both -inf
// here) are no tokens.
__device__ __forceinline__ float logit_of(float l) {
  return l > -__builtin_inff() ? fminf(l, FLT_MAX) : -__builtin_inff();
}
// An integer of the same order, 0 for no token (the key of -inf is 0x007FFFFF).  -0 is
// equal to +0: the sum of both signs' zeros with +0 is +0.
__device__ __forceinline__ uint32_t logit_key(float l) {
  const uint32_t b = __builtin_bit_cast(uint32_t, l + 0.f);
  return l == -__builtin_inff() ? 0u : (b & 0x80000000u) ? ~b : b | 0x80000000u;
}

constexpr int kMassBits = 45;      // a token's p in steps of 2^-45: 2^18 of them fit 64 bits

// p of a logit, and in steps.
__device__ __forceinline__ double mass_of(float l, float top, double inv_t) {
  return exp(((double)l - (double)top) * inv_t);
}
__device__ __forceinline__ uint64_t mass_steps(double p) {
  return (uint64_t)__builtin_rint(p * (double)(1ull << kMassBits));
}

// f * v for 0 <= f, an fp32 number: rounded down or up, not above 2^63.
__device__ __forceinline__ uint64_t scaled(float f, uint64_t v, bool up) {
  if (f >= 1.f) return v;
  const uint32_t b = __builtin_bit_cast(uint32_t, f);
  const int e = (int)(b >> 23);
  const uint64_t mant = e == 0 ? b : (b & 0x7FFFFFu) | 0x800000u;
  const int shift = e == 0 ? 149 : 150 - e;              // f = mant * 2^-shift, shift >= 24
  const unsigned __int128 x = (unsigned __int128)mant * v;
  if (shift >= 128) return up && x != 0;
  const unsigned __int128 q = x >> shift;
  return (uint64_t)q + (up && (q << shift) != x);
}

constexpr int kSampleThreads = 512;
constexpr int kSampleWaves = kSampleThreads / 64;

struct SampleShared {
  uint64_t mass[256];
  uint32_t count[256];
  uint64_t wave_mass[kSampleWaves];
  uint32_t wave_count[kSampleWaves];
  uint32_t digit, above_count;
  uint64_t above_mass;
  int found;
  float tops[kSampleWaves];
};

__device__ __forceinline__ uint64_t shfl_up64(uint64_t v, int d) {
  const uint32_t lo = __shfl_up((uint32_t)v, d), hi = __shfl_up((uint32_t)(v >> 32), d);
  return (uint64_t)hi << 32 | lo;
}

// Sums over the work-group's threads before this one, and over all.
__device__ __forceinline__ void block_scan(SampleShared& sh, uint64_t mass, uint32_t count,
                                           uint64_t& mass_before, uint32_t& count_before,
                                           uint64_t& mass_all, uint32_t& count_all) {
  const int lane = lane_id(), wave = wave_id();
  uint64_t m = mass;
  uint32_t c = count;
  for (int d = 1; d < 64; d *= 2) {
    const uint64_t om = shfl_up64(m, d);
    const uint32_t oc = __shfl_up(c, d);
    if (lane >= d) { m += om; c += oc; }
  }
  if (lane == 63) { sh.wave_mass[wave] = m; sh.wave_count[wave] = c; }
  __syncthreads();
  mass_all = 0;
  count_all = 0;
  mass_before = m - mass;
  count_before = c - count;
  for (int w = 0; w < kSampleWaves; ++w) {
    if (w < wave) { mass_before += sh.wave_mass[w]; count_before += sh.wave_count[w]; }
    mass_all += sh.wave_mass[w];
    count_all += sh.wave_count[w];
  }
  __syncthreads();
}

// One byte of the key, from the highest on, of the token that brings the count or the
// mass of the order's beginning to `need`: the bytes above are `prefix`, tokens above
// them have `count` and `mass`.
template <bool MASS>
__device__ __forceinline__ void select_byte(SampleShared& sh, const float* x, int n, float top,
                                            double inv_t, int shift, uint32_t floor_key,
                                            uint64_t too_much, uint64_t need, uint32_t& prefix,
                                            uint32_t& count, uint64_t& mass) {
  for (int i = threadIdx.x; i < 256; i += kSampleThreads) { sh.count[i] = 0; sh.mass[i] = 0; }
  __syncthreads();
  for (int i = threadIdx.x; i < n; i += kSampleThreads) {
    const float l = logit_of(x[i]);
    const uint32_t key = logit_key(l);
    if (key == 0 || key < floor_key || (shift < 24 && (key >> (shift + 8)) != prefix)) continue;
    const uint32_t d = (key >> shift) & 255u;
    atomicAdd(&sh.count[d], 1u);
    if (MASS) atomicAdd((unsigned long long*)&sh.mass[d],
                        (unsigned long long)mass_steps(mass_of(l, top, inv_t)));
  }
  __syncthreads();
  if (threadIdx.x == 0) {
    uint32_t c = count;
    uint64_t m = mass;
    int d = 255;
    for (;; --d) {
      const uint32_t nc = sh.count[d];
      uint64_t nm = sh.mass[d];
      if (MASS && floor_key != 0 && (prefix << 8 | (uint32_t)d) == floor_key >> shift) nm -= too_much;
      const bool enough = MASS ? m + nm >= need && nc != 0 : c + nc >= need;
      if (enough || d == 0) break;
      c += nc;
      m += nm;
    }
    sh.digit = d;
    sh.above_count = c;
    sh.above_mass = m;
  }
  __syncthreads();
  prefix = shift == 24 ? sh.digit : prefix << 8 | sh.digit;
  count = sh.above_count;
  mass = sh.above_mass;
  __syncthreads();
}

// A row by one work-group, whatever it holds: sums of p are integers (steps of 2^-45), so that
// they do not depend on their order; the last kept token is found byte by byte of its
// logit's bits, over histograms of counts (top_k) and then of masses (top_p).  For rows whose
// cuts lie among more tokens than can be gathered (a flat row: 860 us for 151936 tokens).
__device__ __forceinline__ void sample_alone(const SampleArgs& a, int row, SampleShared& sh) {
  float* tops = sh.tops;
  const int n = a.vocab;
  const float* x = a.logits + row * a.ld;
  SampleRow r = sample_row(a, row);
  float top = -__builtin_inff();
  for (int i = threadIdx.x; i < n; i += kSampleThreads) top = fmaxf(top, logit_of(x[i]));
  for (int d = 32; d > 0; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
  if (lane_id() == 0) tops[wave_id()] = top;
  __syncthreads();
  for (int w = 0; w < kSampleWaves; ++w) top = fmaxf(top, tops[w]);
  if (top == -__builtin_inff()) {
    if (threadIdx.x == 0) {
      a.ids[row] = -1;
      if (a.probs != nullptr) a.probs[row] = 0.f;
    }
    return;
  }
  const bool greedy = r.t == 0.;
  if (greedy) { r.t = 1.; r.k = 0; r.p = 1.f; r.mp = 0.f; r.u = 0.f; }
  const double inv_t = 1. / r.t;
  // the cut: tokens of a key above `cut`, and the first `ties` of those that have it
  uint32_t cut = greedy ? logit_key(top) : 0u, ties = greedy ? 1u : 0xFFFFFFFFu;
  uint64_t too_much = 0;
  if (r.k != 0) {
    uint32_t prefix = 0, count = 0;
    uint64_t mass = 0;
    for (int shift = 24; shift >= 0; shift -= 8)
      select_byte<false>(sh, x, n, top, inv_t, shift, 0u, 0u, (uint64_t)r.k, prefix, count, mass);
    if (count + sh.count[prefix & 255u] >= (uint32_t)r.k) {   // (or there are fewer tokens)
      cut = prefix;
      ties = r.k - count;
      const uint32_t b = cut & 0x80000000u ? cut & 0x7FFFFFFFu : ~cut;
      const float l = __builtin_bit_cast(float, b);
      too_much = (uint64_t)(sh.count[prefix & 255u] - ties) * mass_steps(mass_of(l, top, inv_t));
    }
    __syncthreads();
  }
  if (r.p < 1.f) {
    uint64_t part = 0, before, all;
    uint32_t none, none_all;
    for (int i = threadIdx.x; i < n; i += kSampleThreads) {
      const float l = logit_of(x[i]);
      const uint32_t key = logit_key(l);
      if (key != 0 && key >= cut) part += mass_steps(mass_of(l, top, inv_t));
    }
    block_scan(sh, part, 0u, before, none, all, none_all);
    const uint64_t need = scaled(r.p, all - too_much, true);
    uint32_t prefix = 0, count = 0;
    uint64_t mass = 0;
    for (int shift = 24; shift >= 0; shift -= 8)
      select_byte<true>(sh, x, n, top, inv_t, shift, cut, too_much, need, prefix, count, mass);
    const uint32_t b = prefix & 0x80000000u ? prefix & 0x7FFFFFFFu : ~prefix;
    const uint64_t one = mass_steps(mass_of(__builtin_bit_cast(float, b), top, inv_t));
    const uint64_t rest = need > mass ? need - mass : 0;
    const uint64_t want = one == 0 ? 1 : (rest + one - 1) / one;
    const uint32_t most = cut == prefix ? ties : 0xFFFFFFFFu;
    cut = prefix;
    ties = want < 1 ? 1u : want > most ? most : (uint32_t)want;
  }
  // kept tokens, in the order of the vocabulary: their sum, then the one that is drawn
  uint64_t total = 0;
  for (int pass = 0; pass < 2; ++pass) {
    uint64_t sum = 0;
    uint32_t tied = 0;
    uint64_t need = scaled(r.u, total, false) + 1;
    if (need > total) need = total;
    if (threadIdx.x == 0) sh.found = n;
    __syncthreads();
    for (int base = 0; base < n; base += kSampleThreads) {
      const int i = base + threadIdx.x;
      uint64_t w = 0;
      uint32_t tie = 0;
      if (i < n) {
        const float l = logit_of(x[i]);
        const uint32_t key = logit_key(l);
        if (key != 0 && key >= cut) {
          const double p = mass_of(l, top, inv_t);
          if (l == top || p >= (double)r.mp) {
            w = mass_steps(p);
            tie = key == cut;
          }
        }
      }
      uint64_t wb, wa;
      uint32_t tb, ta;
      block_scan(sh, 0u, tie, wb, tb, wa, ta);
      if (tie && tied + tb >= ties) w = 0;
      tied += ta;
      block_scan(sh, w, 0u, wb, tb, wa, ta);
      if (pass == 1 && w != 0 && sum + wb < need && sum + wb + w >= need) {
        a.ids[row] = i;
        if (a.probs != nullptr) a.probs[row] = (float)((double)w / (double)total);
        sh.found = i;
      }
      sum += wa;
      __syncthreads();
      if (sh.found < n) return;
    }
    total = sum;
    __syncthreads();
  }
}

}  // namespace qlin
