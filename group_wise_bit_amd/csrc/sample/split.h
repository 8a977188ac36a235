// Drawing tokens with a row split over work-groups (gfx950, wave64).
#pragma once

#include "sample.h"

#include <type_traits>

namespace qlin {

// The steps of a draw:
//   bins    every slice of 8192 logits: counts and masses by bins of the exponent,
//   bounds  every row: the bins in which the cuts of top_k, top_p and min_p can lie,
//   gather  every slice: its tokens in these bins, in the order of the vocabulary,
//   pick    every row: the cut among them, the slice that u falls into, the token.
// Exponents are t = 12 l / temperature in 64 bits; a bin is t rounded, so that bins of
// different slices line up whatever their largest logit, and the mass of a
// token is exp((t - bin) / 12), a polynomial of degree 6, times a factor per bin.
// Bins from 384 below the top one (exp(-32)) on hold no mass.
//
// What bounds it.  A logit is read two or three times (the rows of a batch stay in the last
// cache): the floor of 64 rows of 151936 is 7.5 us, of one row nothing.  One row takes four launches
// of 5 to 6 us, each a chain of dependent loads and sums; 64 rows take 18 + 7 + 11 + 20 us: the bins
// are bound by 64-bit arithmetic and an LDS atomic per token, the pick by its chain of
// barriers on 64 CUs.  A row in one work-group (sample_alone) takes 860 us.
constexpr int kSlice = 8192;                 // (4096: 21 us of the bins for 18 at 64 rows)
constexpr int kSlices = 32;                  // of a row, at most
constexpr int kBins = 384;
constexpr int kBinScale = 12;
constexpr int kListMax = 8192;               // tokens that are gathered, at most (what LDS holds)
constexpr int kBinThreads = 512;
// Tokens whose order is found by comparing all, a thread each (one row with top_k 50: 5.5 us of
// the pick, 11.1 through parts).
constexpr int kRankMax = 512;
constexpr int kSums = kBins + 1;             // a slice's sums: 0, then up to each bin

struct SliceStat {
  double top_bin;                          // the bin of its largest logit
  float top;                                 // -inf: no tokens
  int pad;
};

struct RowHead {
  double top_bin;                          // of the row
  float top;
  int mode;                                  // 0: no tokens, 1: largest, 2: list, 3: by itself
  int a, z, e;                               // gathered bins a .. z and e (-1: none)
  int n, main;                               // gathered tokens, those of bins a .. z
  int k_main, k_extra;                       // tokens of a .. z / of e among the first top_k
  double mass_a;                             // of the bins before a
  double mass_k;                             // of the first top_k without those k_main / k_extra
  int slice;                                 // mode 1: the first slice with the largest logit
};
struct RowPlanS {
  RowHead head;
  int at[kSlices + 1];                       // where a slice's tokens begin in the list
  double base[kSlices];                      // a slice's mass of the bins before a
};

struct SplitArgs {
  SampleArgs s;
  int row0, slices;
  double* cum_mass;                          // [rows][slices][kSums]
  uint32_t* cum_count;
  SliceStat* stat;                           // [rows][slices]
  RowPlanS* plan;                            // [rows]
  uint2* list;                               // [rows][kListMax]: index, logit
};

// 12 / temperature in two parts, and t of a logit: hi rounded, lo what is missing.
struct BinScale {
  double hi, lo;
};
__device__ __forceinline__ BinScale bin_scale(double t) {
  BinScale c;
  c.hi = (double)kBinScale / t;
  c.lo = __builtin_fma(-c.hi, t, (double)kBinScale) / t;
  if (!(t < (double)__builtin_inff())) c.lo = 0.;
  return c;
}
__device__ __forceinline__ double t_low(double l, double hi, BinScale c) {
  return __builtin_fma(l, c.lo, __builtin_fma(l, c.hi, -hi));
}
// t less its bin.  From |t| = 2^40 on nothing is left of hi, and lo may be anything: there
// a bin holds one value of l only, and any number will do.
__device__ __forceinline__ double t_rest(double l, double hi, double bin, BinScale c) {
  const double x = (hi - bin) + t_low(l, hi, c);
  return __builtin_fabs(bin) < 0x1p40 ? x : 0.;
}

// exp(x / 12) - 1 + one for |x| <= 1/2 (and a little beyond): x^7 / (12^7 7!) < 2^-44.  The
// coefficients are kept in registers (as constants each would be moved before its fma).
struct MassPoly {
  double c[7];
};
__device__ __forceinline__ MassPoly mass_poly(double one) {
  constexpr double s = 1. / kBinScale;
  MassPoly p{{one, s, s * s / 2, s * s * s / 6, s * s * s * s / 24, s * s * s * s * s / 120,
              s * s * s * s * s * s / 720}};
#pragma unroll
  for (int i = 0; i < 7; ++i) asm("" : "+v"(p.c[i]));
  return p;
}
__device__ __forceinline__ double bin_mass(double x, const MassPoly& k) {
  double p = k.c[6];
#pragma unroll
  for (int i = 5; i >= 0; --i) p = __builtin_fma(p, x, k.c[i]);
  return p;
}
// Masses within a bin are whole numbers of 2^-34: sums of 2^18 equal ones are exact, and
// the sums of histograms and of lists are sums of the same numbers.
constexpr int kMassStep = 34;
constexpr double kMassOne = 1. + (double)(1 << (52 - kMassStep));

// Mass of a logit relative to the middle of the bin `top`, with the factors of the bins from
// there on.
__device__ __forceinline__ double list_mass(float l, double top, BinScale c, const double* factor,
                                            const MassPoly& poly) {
  const double ld = (double)l, hi = ld * c.hi, f = __builtin_rint(hi), k = top - f;
  const double p = bin_mass(t_rest(ld, hi, f, c), poly) - (kMassOne - 1.);
  return k < (double)kBins ? p * factor[(int)k] : 0.;
}
__device__ __forceinline__ double bin_factor(int k) { return exp(-(double)k * (1. / kBinScale)); }
__device__ __forceinline__ int bin_of(float l, double top, BinScale c) {
  const double k = top - __builtin_rint((double)l * c.hi);
  return k < (double)kBins ? (int)k : kBins;
}

template <typename T>
__device__ __forceinline__ T wave_scan(T v) {          // inclusive
  const int lane = lane_id();
  for (int d = 1; d < 64; d *= 2) {
    const T o = __shfl_up(v, d);
    if (lane >= d) v += o;
  }
  return v;
}

// A histogram entry: the count from bit 50 on (8192 at most), the mass in its steps
// below (8192 exp(1 / 24) 2^34 at most): one LDS atomic per token, and a sum that does
// not depend on the order.
constexpr int kCountBit = 50;

// One work-group per slice, 16 logits of a thread in registers: the slice's top first, then
// the histogram, then its sums.
__global__ __launch_bounds__(kBinThreads) void k_sample_bins(const SplitArgs a) {
  __shared__ unsigned long long hist[kBins];
  constexpr int kWaves = kBinThreads / 64;
  __shared__ float tops[kWaves];
  __shared__ double wave_mass[kWaves];
  __shared__ uint32_t wave_count[kWaves];
  const int slice = blockIdx.x % a.slices, r = blockIdx.x / a.slices, row = a.row0 + r;
  const int64_t at = (int64_t)r * a.slices + slice;
  const float* x = a.s.logits + row * a.s.ld + slice * kSlice;
  const int n = min(a.s.vocab - slice * kSlice, kSlice), tid = threadIdx.x, wave = wave_id();
  constexpr int per = kSlice / kBinThreads;
  float l[per];
  float top = -__builtin_inff();
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = j * kBinThreads + tid;
    l[j] = i < n ? x[i] : -__builtin_inff();
  }
  const SampleRow set = sample_row(a.s, row);
  for (int i = tid; i < kBins; i += kBinThreads) hist[i] = 0;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    l[j] = logit_of(l[j]);
    top = fmaxf(top, l[j]);
  }
  for (int d = 32; d > 0; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
  if (lane_id() == 0) tops[wave] = top;
  __syncthreads();
  for (int w = 0; w < kWaves; ++w) top = fmaxf(top, tops[w]);
  const BinScale c = bin_scale(set.t == 0. ? 1. : set.t);
  const double first = top > -__builtin_inff() ? __builtin_rint((double)top * c.hi) : 0.;
  if (tid == 0) {
    a.stat[at] = SliceStat{first, top, 0};
    a.cum_mass[at * kSums] = 0.;
    a.cum_count[at * kSums] = 0;
  }
  if (set.t == 0. || top == -__builtin_inff()) return;
  const MassPoly poly = mass_poly(kMassOne);
  // (a token that is none is infinitely far below)
  auto add = [&](float v, auto far) {
    const double ld = (double)v, hi = ld * c.hi, f = __builtin_rint(hi), k = first - f;
    if (k < (double)kBins) {
      const double t = decltype(far)::value ? t_rest(ld, hi, f, c) : (hi - f) + t_low(ld, hi, c);
      const uint64_t b = __builtin_bit_cast(uint64_t, bin_mass(t, poly));
      atomicAdd(&hist[(int)k], (unsigned long long)((b & ((1ull << 52) - 1)) | (1ull << kCountBit)));
    }
  };
  if (__builtin_fabs(first) < 0x1p39) {        // every bin of the slice is below 2^40
#pragma unroll
    for (int j = 0; j < per; ++j) add(l[j], std::false_type{});
  } else {
#pragma unroll
    for (int j = 0; j < per; ++j) add(l[j], std::true_type{});
  }
  __syncthreads();
  double mass_before = 0.;
  uint32_t count_before = 0;
#pragma unroll
  for (int base = 0; base < kBins; base += kBinThreads) {
    const int k = base + tid;
    const uint64_t h = k < kBins ? hist[k] : 0;
    double m = wave_scan((double)(h & ((1ull << kCountBit) - 1)) * (1. / (double)(1ull << kMassStep)) *
                         bin_factor(k));
    uint32_t q = wave_scan((uint32_t)(h >> kCountBit));
    if (lane_id() == 63) { wave_mass[wave] = m; wave_count[wave] = q; }
    __syncthreads();
    double mb = mass_before;
    uint32_t cb = count_before;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      if (w == wave) { m += mb; q += cb; }
      mb += wave_mass[w];
      cb += wave_count[w];
    }
    mass_before = mb;
    count_before = cb;
    if (k < kBins) {
      a.cum_mass[at * kSums + 1 + k] = m;
      a.cum_count[at * kSums + 1 + k] = q;
    }
    __syncthreads();
  }
}

// One work-group per row, a thread per bin: sums over the slices, 16 slices' loads in flight (with
// a test for each slice they waited for one another: 11 us for 7).
__global__ __launch_bounds__(kBins) void k_sample_bounds(const SplitArgs a) {
  __shared__ double mass[kBins];
  __shared__ uint32_t count[kBins];
  __shared__ double factor[kSlices];
  __shared__ int shift[kSlices];
  const int r = blockIdx.x, row = a.row0 + r, k = threadIdx.x, lane = lane_id();
  RowPlanS& p = a.plan[r];
  const SampleRow set = sample_row(a.s, row);
  const int64_t at = (int64_t)r * a.slices;
  // the row's top, and how far below it the slices begin (every wave by itself)
  const SliceStat st = lane < a.slices ? a.stat[at + lane] : SliceStat{0., -__builtin_inff(), 0};
  float top = st.top;
  for (int d = 32; d > 0; d /= 2) top = fmaxf(top, __shfl_xor(top, d));
  if (top == -__builtin_inff() || set.t == 0.) {
    if (k == 0) {
      p.head.mode = top == -__builtin_inff() ? 0 : 1;
      p.head.top = top;
      p.head.n = 0;
    }
    const uint64_t has = __ballot(st.top == top);
    if (k == 0) p.head.slice = __builtin_ctzll(has);
    return;
  }
  const BinScale c = bin_scale(set.t);
  const double t_top = (double)top * c.hi, f = __builtin_rint(t_top);
  if (k < kSlices) {
    const double d = f - st.top_bin;
    const int s = st.top > -__builtin_inff() && d < (double)kBins ? (int)d : kBins;
    shift[k] = s;
    factor[k] = bin_factor(s);
  }
  __syncthreads();
  double m = 0.;
  uint32_t q = 0;
  constexpr int kFlight = 16;                // slices whose loads are in flight
  for (int s0 = 0; s0 < a.slices; s0 += kFlight) {
    double cm[kFlight];
    uint32_t cq[kFlight];
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      // (a slice without mass in these bins, and one that is not there: its first sum, 0)
      const int64_t i = (at + min(s0 + j, a.slices - 1)) * kSums + max(k + 1 - shift[s0 + j], 0);
      cm[j] = a.cum_mass[i];
      cq[j] = a.cum_count[i];
    }
#pragma unroll
    for (int j = 0; j < kFlight; ++j) {
      m += cm[j] * factor[s0 + j];
      q += cq[j];
    }
  }
  mass[k] = m;
  count[k] = q;
  // the first bin with which the count reaches top_k
  const int bk = set.k != 0 ? __syncthreads_count(q < (uint32_t)set.k) : kBins;
  __syncthreads();
  const bool cut_k = bk < kBins;               // (or fewer tokens have any mass)
  const bool whole = cut_k && count[bk] == (uint32_t)set.k;
  const double all = mass[kBins - 1];
  const double high = cut_k ? mass[bk] : all;
  const double low = !cut_k || whole ? high : bk > 0 ? mass[bk - 1] : 0.;
  // sums of histograms and lists differ by their roundings to 64 bits only
  const bool cut_p = set.p < 1.f;
  const double slack = 1. / (1 << 30);
  const int p0 = __syncthreads_count(m < (double)set.p * low * (1. - slack));
  const int p1 = __syncthreads_count(m < (double)set.p * high * (1. + slack));
  int lo = kBins, hi = kBins;
  if (cut_k) lo = hi = bk;
  if (cut_p) {
    lo = min(lo, min(p0, kBins - 1));
    hi = min(hi, min(p1, kBins - 1));
  }
  if (set.mp > 0.f) {
    const double edge = t_top + log((double)set.mp) * kBinScale;
    const double near = fmax(1. / (1 << 20), __builtin_fabs(t_top) * 0x1p-48);
    const double m0 = f - __builtin_rint(edge + near), m1 = f - __builtin_rint(edge - near);
    lo = min(lo, m0 < (double)kBins ? max((int)m0, 0) : kBins);
    hi = min(hi, m1 < (double)kBins ? max((int)m1, 0) : kBins);
  }
  // (nothing lies beyond the last bin)
  const int last = min(hi, kBins - 1);
  const int extra = cut_p && cut_k && !whole && bk > last ? bk : -1;
  const int more = extra >= 0 ? (int)(count[extra] - count[extra - 1]) : 0;
  // few tokens in all: those before the cuts' bins too, and the draw is made from the list
  const int first = lo < kBins && (int)count[last] + more <= kRankMax ? 0 : lo;
  const uint32_t before = first > 0 ? count[first - 1] : 0u;
  const int main = first < kBins ? (int)(count[last] - before) : 0;
  if (k < 64) {
    // (bins before the slice's first: its first sum, 0)
    const int slice = min(k, a.slices - 1), s = shift[slice];
    const uint32_t* n = a.cum_count + (at + slice) * kSums;
    auto upto = [&](int bin) { return max(bin + 1 - s, 0); };
    const uint32_t n0 = n[upto(first - 1)], n1 = n[upto(last)], n2 = n[upto(extra - 1)],
                   n3 = n[upto(extra)];
    const double before_a = a.cum_mass[(at + slice) * kSums + upto(first - 1)] * factor[slice];
    const int size = k < a.slices ? (first < kBins ? (int)(n1 - n0) : 0) + (extra >= 0 ? (int)(n3 - n2) : 0) : 0;
    const double base = k < a.slices ? before_a : 0.;
    const int end = wave_scan(size);
    if (k < kSlices) {
      p.at[k + 1] = end;
      p.base[k] = base;
    }
    if (k == 0) p.at[0] = 0;
  }
  if (k == 0) {
    p.head.top_bin = f;
    p.head.top = top;
    p.head.a = first;
    p.head.z = last;
    p.head.e = extra;
    p.head.n = main + more;
    p.head.main = main;
    p.head.mode = main + more <= kListMax ? 2 : 3;
    p.head.mass_a = first > 0 ? mass[first - 1] : 0.;
    p.head.k_main = cut_k && bk <= last ? set.k - (int)before : main;
    p.head.k_extra = extra >= 0 ? set.k - (int)count[extra - 1] : 0;
    // the mass of the first top_k: mass_a and the list's, or what lies before the bin e and that bin's
    p.head.mass_k = extra >= 0 ? mass[extra - 1] : cut_k && bk <= last ? -1. : high;
  }
}

// One work-group per slice; a token's place in the list is the number of those before it, so
// that the list has the vocabulary's order.  (Four slices to a work-group: 22 us for 11.)
__global__ __launch_bounds__(kBinThreads) void k_sample_gather(const SplitArgs a) {
  constexpr int kWaves = kBinThreads / 64;
  __shared__ int counts[kSlice / 64];          // [step][wave]
  const int slice = blockIdx.x % a.slices, r = blockIdx.x / a.slices, row = a.row0 + r;
  const RowPlanS& plan = a.plan[r];
  const RowHead p = plan.head;
  const int from = plan.at[slice], to = plan.at[slice + 1];
  const BinScale c = bin_scale(sample_row(a.s, row).t);
  if (p.mode != 2 || from == to) return;
  const float* x = a.s.logits + row * a.s.ld + slice * kSlice;
  const int n = min(a.s.vocab - slice * kSlice, kSlice);
  const double f = p.top_bin;
  const int first = p.a, last = p.z, extra = p.e, lane = lane_id(), wave = wave_id();
  constexpr int per = kSlice / kBinThreads;
  float l[per];
  uint32_t in = 0;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = j * kBinThreads + threadIdx.x;
    l[j] = i < n ? x[i] : -__builtin_inff();
  }
#pragma unroll
  for (int j = 0; j < per; ++j) {
    l[j] = logit_of(l[j]);
    const int k = l[j] > -__builtin_inff() ? bin_of(l[j], f, c) : kBins;
    const bool mine = (k >= first && k <= last) || k == extra;
    in |= (uint32_t)mine << j;
    const uint64_t b = __ballot(mine);
    if (lane == 0) counts[j * kWaves + wave] = __builtin_popcountll(b);
  }
  __syncthreads();
  static_assert(kSlice / 64 == 128, "two counts a lane");
  const int c1 = counts[2 * lane + 1], both = wave_scan(counts[2 * lane] + c1);
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const bool mine = in >> j & 1;
    const uint64_t b = __ballot(mine);
    const int place = j * kWaves + wave, pair = __shfl(both, place / 2), odd = __shfl(c1, place / 2);
    const int end = place % 2 ? pair : pair - odd;
    if (mine) {
      const int pos = from + end - __builtin_popcountll(b) + __builtin_popcountll(b & ((1ull << lane) - 1));
      a.list[(int64_t)r * kListMax + pos] = make_uint2(
          slice * kSlice + j * kBinThreads + threadIdx.x, __builtin_bit_cast(uint32_t, l[j]));
    }
  }
}

constexpr int kPickThreads = kSampleThreads;

// The order of tokens as an ascending integer: by logit, descending, then by index.
__device__ __forceinline__ uint64_t order_key(float l, uint32_t index) {
  return (uint64_t)~logit_key(l) << 32 | index;
}
__device__ __forceinline__ float key_logit(uint64_t key) {
  const uint32_t b = ~(uint32_t)(key >> 32);
  return __builtin_bit_cast(float, b & 0x80000000u ? b & 0x7FFFFFFFu : ~b);
}

// Sorts keys[0 .. size), size a power of two from 64 on: bitonic, exchanges within a wave's 64 keys
// through registers.
__device__ __forceinline__ void sort_keys(uint64_t* keys, int size) {
  for (int k = 2; k <= size; k *= 2) {
    int j = k / 2;
    for (; j >= 64; j /= 2) {
      for (int i = threadIdx.x; i < size / 2; i += kPickThreads) {
        const int lo = 2 * i - (i & (j - 1)), hi = lo + j;
        const uint64_t x = keys[lo], y = keys[hi];
        if ((x > y) == ((lo & k) == 0)) { keys[lo] = y; keys[hi] = x; }
      }
      __syncthreads();
    }
    for (int i = threadIdx.x; i < size; i += kPickThreads) {
      uint64_t x = keys[i];
      for (int d = j; d > 0; d /= 2) {
        const uint32_t ol = __shfl_xor((uint32_t)x, d), oh = __shfl_xor((uint32_t)(x >> 32), d);
        const uint64_t y = (uint64_t)oh << 32 | ol;
        const bool lower = (i & d) == 0, up = (i & k) == 0;
        x = (lower == up) == (x < y) ? x : y;
      }
      keys[i] = x;
    }
    __syncthreads();
  }
}

// The gathered tokens are sorted into 1024 parts of their range, by t: bins a .. z share kMainParts
// of them, the bin e has the rest.  Counts and masses of the parts tell where a cut lies; only the
// tokens of that part are put in order.  Masses are whole numbers of 2^-50 of bin a's (or e's)
// unit, so that a sum does not depend on its order: 8192 tokens, exp(1 / 24) at most each, stay below
// 2^64, and a token far below bin a's is off by 2^-51 of the unit (the sum over all kept ones,
// the largest logit's among them, is 0.95 units at least).
constexpr int kParts = 1024;
constexpr int kMainParts = 896;
constexpr int kPartStep = 50;
static_assert(kListMax <= 1 << (63 - kPartStep), "sums of parts");

struct PickShared {
  float l[kListMax];                         // the gathered tokens
  uint32_t index[kListMax];
  uint16_t part_of[kListMax];
  uint64_t keys[kListMax];                   // a part's tokens in order
  unsigned long long part[kParts];           // masses up to a part
  uint32_t part_count[kParts];               // tokens up to a part
  double factor[kBins];
  unsigned long long slice_mass[kSlices];
  double wave[kSampleWaves];
  uint64_t scan[kSampleWaves];
  uint32_t scan_count[kSampleWaves];
  double before, target, total;
  uint64_t cut;
  int slice, count[3], size, at, rank;
};

// Sums of v over the threads up to this one; over all in sh.total.
__device__ __forceinline__ double sum_before(PickShared& sh, double v) {
  const int wave = wave_id();
  double up = wave_scan(v), all = 0.;
  if (lane_id() == 63) sh.wave[wave] = up;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kSampleWaves; ++w) {
    if (w == wave) up += all;
    all += sh.wave[w];
  }
  if (threadIdx.x == 0) sh.total = all;
  __syncthreads();
  return up;
}

// The tokens of a part in order: sh.keys[0 .. sh.size).
__device__ __forceinline__ void order_part(PickShared& sh, int n, int part) {
  if (threadIdx.x == 0) sh.size = 0;
  __syncthreads();
#pragma unroll 1
  for (int i = threadIdx.x; i < n; i += kPickThreads)
    if (sh.part_of[i] == part) sh.keys[atomicAdd(&sh.size, 1)] = order_key(sh.l[i], sh.index[i]);
  __syncthreads();
  const int m = sh.size;
  if (m <= kPickThreads) {
    // a token's place is the number of those before it
    const int i = threadIdx.x;
    const uint64_t mine = i < m ? sh.keys[i] : 0;
    int rank = 0;
    if (wave_id() * 64 < m)
#pragma unroll 4
      for (int j = 0; j < m; ++j) rank += sh.keys[j] < mine;
    __syncthreads();
    if (i < m) sh.keys[rank] = mine;
    __syncthreads();
    return;
  }
  int size = 64;
  while (size < m) size *= 2;
  for (int i = m + threadIdx.x; i < size; i += kPickThreads) sh.keys[i] = ~0ull;
  __syncthreads();
  sort_keys(sh.keys, size);
}

// The first part whose sum (counts or masses, from `from` on) reaches `need`; kParts: none.
template <typename F>
__device__ __forceinline__ int first_part(PickShared& sh, int from, int to, F reaches) {
  if (threadIdx.x == 0) sh.at = kParts;
  __syncthreads();
#pragma unroll 1
  for (int i = from + threadIdx.x; i < to; i += kPickThreads)
    if (reaches(i) && (i == from || !reaches(i - 1))) sh.at = i;
  __syncthreads();
  return sh.at;
}

// Mass of the first `rank` ordered tokens, in the units of list_mass.
__device__ __forceinline__ double mass_of_first(PickShared& sh, int rank, double f, BinScale c,
                                                const MassPoly& poly) {
  double s = 0.;
  for (int i = threadIdx.x; i < rank; i += kPickThreads) s += list_mass(key_logit(sh.keys[i]), f, c, sh.factor, poly);
  for (int d = 32; d > 0; d /= 2) s += __shfl_xor(s, d);
  if (lane_id() == 0) sh.wave[wave_id()] = s;
  __syncthreads();
  s = 0.;
  for (int w = 0; w < kSampleWaves; ++w) s += sh.wave[w];
  __syncthreads();
  return s;
}

// How many of the ordered tokens it takes until `sum` and their masses reach `target` (all of
// them if they do not; 1 at least).
__device__ __forceinline__ int first_to_reach(PickShared& sh, double sum, double target, double f,
                                              BinScale c, const MassPoly& poly) {
  const int n = sh.size, wave = wave_id();
  if (threadIdx.x == 0) sh.rank = n > 0 ? n : 1;
  __syncthreads();
  for (int base = 0; base < n; base += kPickThreads) {
    const int i = base + threadIdx.x;
    const double up = wave_scan(i < n ? list_mass(key_logit(sh.keys[i]), f, c, sh.factor, poly) : 0.);
    if (lane_id() == 63) sh.wave[wave] = up;
    __syncthreads();
    double run = sum + up;
    for (int w = 0; w < kSampleWaves; ++w) {
      if (w < wave) run += sh.wave[w];
      sum += sh.wave[w];
    }
    if (i < n && run >= target) atomicMin(&sh.rank, i + 1);
    __syncthreads();
    if (sum >= target) break;
  }
  return sh.rank;
}

// One work-group per row.  The cut is put together as top_k, then top_p of the first top_k's
// mass, then min_p; the draw goes through the slices' masses to one slice's logits, or, where all
// kept tokens are in the list, through the list alone.
__global__ __launch_bounds__(kPickThreads) void k_sample_pick(const SplitArgs a) {
  __shared__ PickShared sh;
  const int r = blockIdx.x, row = a.row0 + r, lane = lane_id(), tid = threadIdx.x;
  const RowPlanS& plan = a.plan[r];
  const RowHead p = plan.head;
  const SampleRow set = sample_row(a.s, row);
  const float* x = a.s.logits + row * a.s.ld;
  const int mode = p.mode;
  if (mode == 3) {
    sample_alone(a.s, row, reinterpret_cast<SampleShared&>(sh));
    return;
  }
  if (mode == 0) {
    if (tid == 0) {
      a.s.ids[row] = -1;
      if (a.s.probs != nullptr) a.s.probs[row] = 0.f;
    }
    return;
  }
  if (mode == 1) {
    if (tid == 0) sh.slice = 0x7FFFFFFF;
    __syncthreads();
    for (int i = p.slice * kSlice + tid; i < min((p.slice + 1) * kSlice, a.s.vocab); i += kPickThreads)
      if (logit_of(x[i]) == p.top) atomicMin(&sh.slice, i);
    __syncthreads();
    if (tid == 0) {
      a.s.ids[row] = sh.slice;
      if (a.s.probs != nullptr) a.s.probs[row] = 1.f;
    }
    return;
  }
  const double base = plan.base[min(lane, a.slices - 1)];
  const BinScale c = bin_scale(set.t);
  const double f = p.top_bin;
  const MassPoly poly = mass_poly(kMassOne);
  const int n = p.n, main = p.main;
  const uint2* list = a.list + (int64_t)r * kListMax;
  uint64_t cut = 0;                            // keys up to it are kept
  constexpr double kStep = 1. / (double)(1ull << kPartStep);
  const double top_hi = (double)p.top * c.hi, top_lo = t_low((double)p.top, top_hi, c);
  // p of a token relative to the largest one's
  auto relative = [&](float l) {
    const double hi = (double)l * c.hi;
    return exp((hi - top_hi + (t_low((double)l, hi, c) - top_lo)) * (1. / kBinScale));
  };
  if (n > 0 && n <= kRankMax) {
    // a token per thread, and its place in the order
    const uint2 t = tid < n ? list[tid] : make_uint2(0, 0);
    const float l = __builtin_bit_cast(float, t.y);
    const uint64_t key = order_key(l, t.x);
    if (tid < n) sh.keys[tid] = key;
    __syncthreads();
    int rank = 0;
    double m = 0.;
    if (wave_id() * 64 < n) {
#pragma unroll 8
      for (int j = 0; j < n; ++j) rank += sh.keys[j] < key;
      const double ld = (double)l, hi = ld * c.hi, bin = __builtin_rint(hi);
      m = (bin_mass(t_rest(ld, hi, bin, c), poly) - (kMassOne - 1.)) * bin_factor((int)(f - bin));
    }
    __syncthreads();
    double* const sums = reinterpret_cast<double*>(sh.keys);      // of the order's first tokens
    if (tid < n) sums[rank] = m;
    __syncthreads();
    const double up = sum_before(sh, tid < n ? sums[tid] : 0.);
    if (tid < n) sums[tid] = up;
    __syncthreads();
    int kept = p.k_main;
    if (set.p < 1.f) {
      const double mass_k = p.e >= 0 ? p.mass_k + sums[main + p.k_extra - 1] - (main > 0 ? sums[main - 1] : 0.)
                            : p.mass_k < 0. ? p.mass_a + sums[p.k_main - 1] : p.mass_k;
      const double target = (double)set.p * mass_k;
      kept = min(kept, 1 + __syncthreads_count(tid < main && p.mass_a + sums[tid] < target));
    }
    if (set.mp > 0.f)
      kept = min(kept, __syncthreads_count(tid < n && rank < main &&
                                           (l == p.top || relative(l) >= (double)set.mp)));
    const bool mine = tid < n && rank < kept;
    if (p.a == 0) {
      // all kept tokens are here, in the order of the vocabulary
      const double w = mine ? m : 0., end = sum_before(sh, w), total = sh.total;
      const bool past = mine && end > (double)set.u * total;
      if (tid == 0) {
        sh.count[0] = 0x7FFFFFFF;
        sh.count[1] = -1;
      }
      __syncthreads();
      const uint64_t hits = __ballot(past), tails = __ballot(mine);
      if (lane == 0 && hits != 0) atomicMin(&sh.count[0], tid + __builtin_ctzll(hits));
      if (lane == 0 && tails != 0) atomicMax(&sh.count[1], tid + 63 - __builtin_clzll(tails));
      __syncthreads();
      // (every p is above 0 here: the last one is that of a u near 1)
      if (tid == min(sh.count[0], sh.count[1])) {
        a.s.ids[row] = t.x;
        if (a.s.probs != nullptr) a.s.probs[row] = (float)(w / total);
      }
      return;
    }
    if (tid < kSlices) sh.slice_mass[tid] = 0;
    if (tid < kBins) sh.factor[tid] = bin_factor(tid);
    if (mine && rank == kept - 1) sh.cut = key;
    __syncthreads();
    if (kept > 0) cut = sh.cut;
    if (mine) atomicAdd(&sh.slice_mass[t.x / kSlice],
                        (unsigned long long)__builtin_rint(m / (sh.factor[p.a] * kStep)));
  } else {
    if (tid < kSlices) sh.slice_mass[tid] = 0;
    if (tid < kBins) sh.factor[tid] = bin_factor(tid);
  }
  __syncthreads();
  const double to_mass = p.a < kBins ? sh.factor[p.a] * kStep : 0.;   // bin a's
  if (n > kRankMax) {
    for (int i = tid; i < kParts; i += kPickThreads) {
      sh.part[i] = 0;
      sh.part_count[i] = 0;
    }
    __syncthreads();
    const double scale = (double)kMainParts / (double)(p.z + 1 - p.a);
    // part and steps of a token
    auto place = [&](float l, uint64_t& steps) {
      const double ld = (double)l, hi = ld * c.hi, bin = __builtin_rint(hi);
      const double x = t_rest(ld, hi, bin, c);                  // in the bin, about -1/2 .. 1/2
      const int k = (int)(f - bin);
      const bool extra = k > p.z;
      const double y = __builtin_fmin(__builtin_fmax(0.5 - x, 0.), 1.);
      double rel = bin_mass(x, poly) - (kMassOne - 1.);
      if (!extra) rel *= sh.factor[k - p.a];
      steps = (uint64_t)__builtin_rint(rel * (double)(1ull << kPartStep));
      return extra ? kMainParts + min((int)(y * (kParts - kMainParts)), kParts - kMainParts - 1)
                   : min((int)(((double)(k - p.a) + y) * scale), kMainParts - 1);
    };
    // (the next two tokens' loads are in flight while one is placed)
    uint2 w0 = list[min(tid, n - 1)], w1 = list[min(tid + kPickThreads, n - 1)];
#pragma unroll 1
    for (int i = tid; i < n; i += kPickThreads) {
      const uint2 w2 = list[min(i + 2 * kPickThreads, n - 1)];
      const float l = __builtin_bit_cast(float, w0.y);
      uint64_t steps;
      const int part = place(l, steps);
      sh.l[i] = l;
      sh.index[i] = w0.x;
      sh.part_of[i] = (uint16_t)part;
      atomicAdd(&sh.part[part], (unsigned long long)steps);
      atomicAdd(&sh.part_count[part], 1u);
      w0 = w1;
      w1 = w2;
    }
    __syncthreads();
    // sums up to a part; the bin e's begin anew
    static_assert(kParts == 2 * kPickThreads && kMainParts % 128 == 0, "two parts a thread");
    {
      const uint64_t v0 = sh.part[2 * tid], v1 = sh.part[2 * tid + 1];
      const uint32_t c0 = sh.part_count[2 * tid], c1 = sh.part_count[2 * tid + 1];
      uint64_t v = v0 + v1;
      uint32_t q = c0 + c1;
      for (int d = 1; d < 64; d *= 2) {
        const uint64_t ov = shfl_up64(v, d);
        const uint32_t oq = __shfl_up(q, d);
        if (lane >= d) { v += ov; q += oq; }
      }
      if (lane == 63) { sh.scan[wave_id()] = v; sh.scan_count[wave_id()] = q; }
      __syncthreads();
      for (int w = 2 * tid >= kMainParts ? kMainParts / 128 : 0; w < wave_id(); ++w) {
        v += sh.scan[w];
        q += sh.scan_count[w];
      }
      sh.part[2 * tid] = v - v1;
      sh.part[2 * tid + 1] = v;
      sh.part_count[2 * tid] = q - c1;
      sh.part_count[2 * tid + 1] = q;
      __syncthreads();
    }
    auto count_to = [&](int part, int from) { return part > from ? (int)sh.part_count[part - 1] : 0; };
    auto mass_to = [&](int part, int from) { return part > from ? (double)sh.part[part - 1] : 0.; };
    // tokens of a .. z that are kept: the first `kept` of them in order
    int kept = p.k_main;
    int held = -1;                             // part of a .. z that sh.keys holds
    auto rank_of = [&](int want) {             // the want-th token is sh.keys[rank_of(want) - 1]
      if (held < 0 || want <= count_to(held, 0) || want > count_to(held, 0) + sh.size) {
        held = first_part(sh, 0, kMainParts, [&](int i) { return (int)sh.part_count[i] >= want; });
        order_part(sh, n, held);
      }
      return want - count_to(held, 0);
    };
    if (set.p < 1.f) {
      double mass_k = p.mass_k;
      if (p.e >= 0) {
        const int pe = first_part(sh, kMainParts, kParts,
                                  [&](int i) { return (int)sh.part_count[i] >= p.k_extra; });
        order_part(sh, n, pe);
        mass_k += mass_to(pe, kMainParts) * sh.factor[p.e] * kStep +
                  mass_of_first(sh, p.k_extra - count_to(pe, kMainParts), f, c, poly);
      } else if (mass_k < 0.) {
        const int rank = rank_of(p.k_main);
        mass_k = p.mass_a + mass_to(held, 0) * to_mass + mass_of_first(sh, rank, f, c, poly);
      }
      // the token with which the sum reaches the target (by rounding there may be none: all)
      const double target = (double)set.p * mass_k;
      const int pp = first_part(sh, 0, kMainParts, [&](int i) {
        return p.mass_a + (double)sh.part[i] * to_mass >= target; });
      if (pp < kParts && count_to(pp, 0) < kept) {
        if (held != pp) order_part(sh, n, pp);
        held = pp;
        kept = min(kept, count_to(pp, 0) + first_to_reach(sh, p.mass_a + mass_to(pp, 0) * to_mass,
                                                          target, f, c, poly));
      }
    }
    if (set.mp > 0.f) {
      int pass = 0;
#pragma unroll 1
      for (int i = tid; i < n; i += kPickThreads)
        if (sh.part_of[i] < kMainParts)
          pass += sh.l[i] == p.top || relative(sh.l[i]) >= (double)set.mp;
      for (int d = 32; d > 0; d /= 2) pass += __shfl_xor(pass, d);
      if (threadIdx.x == 0) sh.count[0] = 0;
      __syncthreads();
      if (lane == 0 && pass) atomicAdd(&sh.count[0], pass);
      __syncthreads();
      kept = min(kept, sh.count[0]);
    }
    if (kept >= main) cut = ~0ull;             // all of a .. z
    else if (kept > 0) cut = sh.keys[rank_of(kept) - 1];
    __syncthreads();
    // the kept ones' masses, slice by slice
#pragma unroll 1
    for (int i = tid; i < n; i += kPickThreads)
      if (sh.part_of[i] < kMainParts && order_key(sh.l[i], sh.index[i]) <= cut) {
        uint64_t steps;
        place(sh.l[i], steps);
        atomicAdd(&sh.slice_mass[sh.index[i] / kSlice], (unsigned long long)steps);
      }
  }
  __syncthreads();
  // the slice that u falls into
  if (wave_id() == 0) {
    double w = 0.;
    if (lane < a.slices) {
      w = base + (double)sh.slice_mass[lane] * to_mass;
    }
    const double end = wave_scan(w);
    const double total = __shfl(end, 63), target = (double)set.u * total;
    const uint64_t past = __ballot(w > 0. && end > target), any = __ballot(w > 0.);
    const int s = past != 0 ? __builtin_ctzll(past) : 63 - __builtin_clzll(any);
    if (lane == s) {
      sh.slice = s;
      sh.before = end - w;
      sh.target = target;
      sh.total = total;
      sh.count[0] = sh.count[1] = 0x7FFFFFFF;
      sh.count[2] = -1;
    }
  }
  __syncthreads();
  // the token in the slice: its logits through LDS, a thread's `per` of them in a row
  constexpr int per = kSlice / kPickThreads;
  const int first = sh.slice * kSlice, i0 = first + tid * per;
  float* const logits = reinterpret_cast<float*>(sh.keys);
  static_assert((kSlice + kPickThreads) * sizeof(float) <= sizeof(sh.keys), "a slice");
#pragma unroll
  for (int j = 0; j < per; ++j) {
    const int i = j * kPickThreads + tid;
    logits[i + i / per] = first + i < a.s.vocab ? x[first + i] : -__builtin_inff();
  }
  __syncthreads();
  const int limit = cut == 0 ? p.a : p.z + 1;
  double w[per], s = 0.;
#pragma unroll
  for (int j = 0; j < per; ++j) {
    w[j] = 0.;
    const float l = logit_of(logits[tid * (per + 1) + j]);
    // (tokens of the bins before a come before any of the list)
    const bool in = cut != 0 && cut != ~0ull ? order_key(l, i0 + j) <= cut
                                             : l > -__builtin_inff() && bin_of(l, f, c) < limit;
    if (in) w[j] = list_mass(l, f, c, sh.factor, poly);
    s += w[j];
  }
  const double up = wave_scan(s);
  if (lane == 63) sh.wave[wave_id()] = up;
  __syncthreads();
  double run = sh.before + (up - s);
  for (int v = 0; v < wave_id(); ++v) run += sh.wave[v];
  int hit = 0x7FFFFFFF, tail = -1;             // the first beyond the target, the last of all
#pragma unroll
  for (int j = 0; j < per; ++j) {
    run += w[j];
    if (w[j] > 0.) {
      if (run > sh.target) hit = min(hit, i0 + j);
      tail = i0 + j;
    }
  }
  for (int d = 32; d > 0; d /= 2) {
    hit = min(hit, __shfl_xor(hit, d));
    tail = max(tail, __shfl_xor(tail, d));
  }
  if (lane == 0) {
    atomicMin(&sh.count[0], hit);
    atomicMax(&sh.count[2], tail);
  }
  __syncthreads();
  const int id = sh.count[0] != 0x7FFFFFFF ? sh.count[0] : sh.count[2];
#pragma unroll
  for (int j = 0; j < per; ++j)
    if (i0 + j == id) {
      a.s.ids[row] = id;
      if (a.s.probs != nullptr) a.s.probs[row] = (float)(w[j] / sh.total);
    }
}

}  // namespace qlin
