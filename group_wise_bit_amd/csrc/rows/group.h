// Kernels beside the row-wise products that no bit width changes: grouping rows
// by expert, the sum over a token's experts, the adapters' first product.
#pragma once

#include "rows.h"

namespace qlin {

// ------------------------------------------------------------ grouping rows --
// A stable counting sort of `count` ids: positions 0 .. count-1 hold the
// indexes of the ids, bucket after bucket, in order within a bucket; ids
// outside [0, buckets) share a last bucket.  Also the table of row tiles: up
// to `rows` positions of one bucket each.  A work-group takes a share of the ids
// (few ids: all of them), wave w the w-th 16th of it, counted in counters of its
// own; the counters are turned into starts, and a second pass writes the
// positions, 64 ids at a time: each lane sets its bit in its bucket's mask, and the
// bits below its own are the equal ids before it.  The atomics (LDS, one wave's)
// count and OR, so the order is the ids' own.  (Masks by ballots over the id's bits took 60 of
// 90 instructions per 64 ids: one work-group took 29 us for 16384 ids over 32
// buckets; with the masks 18 us.)  Beyond kPlanIds the ids are shared out, each
// work-group's counts having been written by k_rows_count before: 8192 ids take 6.9
// us in one work-group, 16384 18 us and shared 7.7, 65536 shared 10.
constexpr int kPlanWaves = 16;
constexpr int kPlanIds = 8192;
constexpr int kPlanGroups = 64;          // work-groups at most

// Ids of a work-group's share (count: of all).
__host__ __device__ inline int plan_share(int count) {
  if (count <= kPlanIds) return count;
  const int groups = count / 1024 < kPlanGroups ? count / 1024 : kPlanGroups;
  return ((count + groups - 1) / groups + 1023) / 1024 * 1024;
}

// Sum of v over the lanes below this one.
__device__ __forceinline__ int lanes_before(int v) {
  int s = v;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int o = __shfl_up(s, d);
    if (lane_id() >= d) s += o;
  }
  return s - v;
}

// Inclusive sums of a and b over the 1024 threads of the work-group (thread
// order), each with the group's total; part is scratch.
__device__ __forceinline__ void group_scan2(int& a, int& b, int (*part)[2]) {
  const int lane = lane_id(), wave = wave_id();
  int ia = lanes_before(a) + a, ib = lanes_before(b) + b;
  if (lane == 63) { part[wave][0] = ia; part[wave][1] = ib; }
  __syncthreads();
  for (int w = 0; w < wave; ++w) { ia += part[w][0]; ib += part[w][1]; }
  a = ia;
  b = ib;
}

// Orders a wave's accesses to its own LDS counters between lanes (a wave's LDS
// instructions execute in order; this keeps the compiler from moving them).
__device__ __forceinline__ void counters_written() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// counts[work-group][bucket] of the shares, bucket `buckets` the ids outside.
__global__ __launch_bounds__(1024) void k_rows_count(const int32_t* __restrict__ ids, int count,
                                                     int buckets, int32_t* __restrict__ counts) {
  __shared__ int hist[kMaxExperts + 1];
  for (int i = threadIdx.x; i <= buckets; i += 1024) hist[i] = 0;
  __syncthreads();
  const int share = plan_share(count);
  const int64_t i0 = (int64_t)blockIdx.x * share;
  const int end = (int)min((int64_t)count, i0 + share);
  for (int i = (int)i0 + threadIdx.x; i < end; i += 1024) {
    const int id = ids[i];
    atomicAdd(&hist[(uint32_t)id < (uint32_t)buckets ? id : buckets], 1);
  }
  __syncthreads();
  for (int i = threadIdx.x; i <= buckets; i += 1024)
    counts[(int64_t)blockIdx.x * (buckets + 1) + i] = hist[i];
}

// counts: of the shares, or null where one work-group takes all ids.
__global__ __launch_bounds__(kPlanWaves * 64) void k_rows_plan(
    const int32_t* __restrict__ ids, int count, int buckets, int rows,
    const int32_t* __restrict__ counts, RowPlan plan) {
  __shared__ int hist[kPlanWaves][kMaxExperts + 1];
  __shared__ unsigned long long mask[kPlanWaves][kMaxExperts + 1];
  __shared__ int part[kPlanWaves][2];
  __shared__ int2 first[kMaxExperts + 1];    // each bucket's first tile and position
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  for (int i = lane; i <= buckets; i += 64) {
    hist[wave][i] = 0;
    mask[wave][i] = 0;
  }
  counters_written();
  const int all = plan_share(count);
  const int g0 = blockIdx.x * all, g1 = min(count, g0 + all);   // (the last share starts below count)
  const int share = ((g1 - g0 + kPlanWaves * 64 - 1) / (kPlanWaves * 64)) * 64;
  const int i0 = min(g1, g0 + wave * share), i1 = min(g1, i0 + share);
  // the buckets of 8 x 64 ids, loaded together
  constexpr int U = 8;
  int id8[U];
  auto load_ids = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = b + 64 * u + lane;
      const int id = i < i1 ? ids[i] : 0;
      id8[u] = (uint32_t)id < (uint32_t)buckets ? id : buckets;
    }
  };
  for (int b0 = i0; b0 < i1; b0 += 64 * U) {
    load_ids(b0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (b0 + 64 * u + lane < i1) atomicAdd(&hist[wave][id8[u]], 1);
    }
  }
  __syncthreads();
  // thread t: bucket t's count, starts of its waves, its start and its tiles'; the
  // ids of earlier shares come first in it
  int total = 0, earlier = 0, before[kPlanWaves];
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) before[w] = tid <= buckets ? hist[w][tid] : 0;
#pragma unroll
  for (int w = 0; w < kPlanWaves; ++w) {
    const int c = before[w];
    before[w] = total;
    total += c;
  }
  if (counts != nullptr && tid <= buckets) {
    total = 0;
    const int groups = gridDim.x;
    for (int b = 0; b < groups; b += 16) {
      int c[16];
#pragma unroll
      for (int g = 0; g < 16; ++g) c[g] = counts[min(b + g, groups - 1) * (buckets + 1) + tid];
#pragma unroll
      for (int g = 0; g < 16; ++g) {
        if (b + g < groups) total += c[g];
        if (b + g < (int)blockIdx.x) earlier += c[g];
      }
    }
  }
  const int mine = tid < buckets ? (total + rows - 1) / rows : 0;
  int end = total, tend = mine;
  group_scan2(end, tend, part);
  const int start = end - total;
  if (tid <= buckets) {
#pragma unroll
    for (int w = 0; w < kPlanWaves; ++w) hist[w][tid] = start + earlier + before[w];
    if (tid == buckets && blockIdx.x == 0) *plan.ntiles = tend;
    first[tid] = make_int2(tend - mine, start);
  }
  __syncthreads();
  // tile i belongs to the last bucket that starts at or before it
  const int ntiles = first[buckets].x;
  for (int i = blockIdx.x * kPlanWaves * 64 + tid; i < ntiles; i += gridDim.x * kPlanWaves * 64) {
    int lo = 0, hi = buckets;
    while (hi - lo > 1) {
      const int mid = (lo + hi) / 2;
      if (first[mid].x <= i) lo = mid;
      else hi = mid;
    }
    const int p0 = first[lo].y + (i - first[lo].x) * rows;
    plan.tiles[i] = make_int4(lo, p0, min(rows, first[lo + 1].y - p0), 0);
  }
  const bool kept = i1 - i0 <= 64 * U;       // the first pass's ids are all of the wave's
  for (int b0 = i0; b0 < i1; b0 += 64 * U) {
    if (!kept) load_ids(b0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int b = b0 + 64 * u, id = id8[u];
      if (b >= i1) break;
      const bool in = b + lane < i1;
      if (in) atomicOr(&mask[wave][id], 1ull << lane);
      counters_written();
      const uint64_t m = mask[wave][id];
      const int below = __builtin_popcountll(m & ((1ull << lane) - 1));
      int at = 0;
      if (in) {
        at = hist[wave][id] + below;
        plan.order[at] = b + lane;
      }
      counters_written();
      if (in && below == 0) {
        hist[wave][id] = at + __builtin_popcountll(m);
        mask[wave][id] = 0;
      }
      counters_written();
    }
  }
}

// ------------------------------------------------- sum over a token's experts --
// Y[i, :] = the rows of its valid (token, slot) pairs, added in slot order.
// One thread: 4 columns of one token (n is a multiple of 64), the rows of 8
// slots requested together.  Bound by the fp32 rows' bytes: 4 slots of 4096 tokens
// of 2048 columns, 151 MB, 22 us (6.9 TB/s: part of them is still in the caches).
__global__ __launch_bounds__(256) void k_rows_combine(
    const float* __restrict__ d, const int32_t* __restrict__ ids, int m, int top_k, int experts,
    int n, float* __restrict__ y, uint16_t* __restrict__ y16, int64_t ldy) {
  const int n4 = n / 4;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < (int64_t)m * n4;
       q += (int64_t)gridDim.x * 256) {
    const int64_t i = q / n4;
    const int c = (int)(q % n4) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    constexpr int U = 8;
    for (int j0 = 0; j0 < top_k; j0 += U) {
      f32x4 v[U];
      int id[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t p = i * top_k + min(j0 + u, top_k - 1);
        id[u] = ids[p];
        v[u] = *reinterpret_cast<const f32x4*>(d + p * n + c);
      }
#pragma unroll
      for (int u = 0; u < U; ++u)     // (rows of pairs without an expert are not written: any bits)
        if (j0 + u < top_k && (uint32_t)id[u] < (uint32_t)experts) s += v[u];
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (y != nullptr) y[i * ldy + c + e] = s[e];
      if (y16 != nullptr) y16[i * ldy + c + e] = __builtin_bit_cast(uint16_t, (f16)s[e]);
    }
  }
}

// ------------------------------------------------------ A x of the adapters --
struct ShrinkArgs {
  const uint16_t* X;
  int64_t ldx;
  int m, k, slots, rank, rp;
  const int32_t* ids;
  const uint16_t* a;      // [slots][rank][k]
  const float* scale;     // [slots] or null
  float* t;               // [splits][m][rp]
  RowPlan plan;           // (tile form) rows by adapter, 16 at a time
  int splits, steps;      // (tile form) K splits; 128-column steps per split
};

__device__ __forceinline__ float dot8(uint4 x, uint4 y, float s) {
  s = __builtin_amdgcn_fdot2(as_h2(x.x), as_h2(y.x), s, false);
  s = __builtin_amdgcn_fdot2(as_h2(x.y), as_h2(y.y), s, false);
  s = __builtin_amdgcn_fdot2(as_h2(x.z), as_h2(y.z), s, false);
  return __builtin_amdgcn_fdot2(as_h2(x.w), as_h2(y.w), s, false);
}

// Few rows, each with an adapter of its own: one wave per (row, rank row), with
// the loads of 4096 columns in flight together.  grid = (m, ceil(rp / 8)).
__global__ __launch_bounds__(512) void k_lora_shrink_row(const ShrinkArgs s) {
  const int lane = lane_id();
  const int64_t row = blockIdx.x;
  const int r = blockIdx.y * 8 + wave_id();
  const int slot = s.ids[row];
  if ((uint32_t)slot >= (uint32_t)s.slots || r >= s.rp) return;
  float sum = 0.f;
  if (r < s.rank) {
    const uint16_t* x = s.X + row * s.ldx;
    const uint16_t* ar = s.a + ((int64_t)slot * s.rank + r) * s.k;
    constexpr int U = 8;
    float part[2] = {0.f, 0.f};
    for (int k0 = 8 * lane; k0 < s.k; k0 += 512 * U) {
      uint4 av[U], xv[U];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const bool in = k0 + 512 * u < s.k;
        const int k = in ? k0 + 512 * u : k0;
        av[u] = *reinterpret_cast<const uint4*>(ar + k);
        xv[u] = *reinterpret_cast<const uint4*>(x + k);
        if (!in) av[u] = xv[u] = make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < U; ++u) part[u & 1] = dot8(av[u], xv[u], part[u & 1]);
    }
    sum = row_sum16(part[0] + part[1]);
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (s.scale != nullptr) sum *= s.scale[slot];
  }
  if (lane == 0) s.t[row * s.rp + r] = sum;
}

// Many rows, ordered by adapter: one work-group per 16 rows of one adapter and
// K split.  v_mfma_f32_16x16x32_f16: lane (c, q) supplies row c of X and rank
// row 16 i + c of A at K positions 8q .. +7 of each 32; the 8 waves take
// 128-column steps in turn and add their sums in LDS in wave order.  Bound by the
// first reads of A and X: the tiles of one adapter go to one XCD, which brought
// 2048 rows of rank 64 and 8 adapters of 4096 columns from 22 to 15 us (32 rows
// per work-group, half of the reads of A: 16 us; 4 splits of K for 2 cost the
// product that adds them 5 us).
template <int NR>
__global__ __launch_bounds__(512) void k_lora_shrink_tile(const ShrinkArgs s) {
  __shared__ f32x4 red[8][NR][64];
  const int total = *s.plan.ntiles * s.splits;
  if ((int)blockIdx.x >= total) return;
  const int at = xcd_position(total), sp = at % s.splits;
  const int4 tile = s.plan.tiles[at / s.splits];
  const int slot = tile.x, p0 = tile.y, rows = tile.z;
  const int lane = lane_id(), wave = wave_id();
  const int c = lane & 15, q = lane >> 4;
  const uint16_t* x = s.X + (int64_t)s.plan.order[p0 + (c < rows ? c : 0)] * s.ldx + 8 * q;
  const uint16_t* ar[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i)
    ar[i] = s.a + ((int64_t)slot * s.rank + min(16 * i + c, s.rank - 1)) * s.k + 8 * q;
  f32x4 acc[NR];
#pragma unroll
  for (int i = 0; i < NR; ++i) acc[i] = (f32x4){0.f, 0.f, 0.f, 0.f};
  const int end = min(s.k, (sp + 1) * s.steps * 128);
  for (int k = (sp * s.steps + wave) * 128; k < end; k += 8 * 128) {
    f16x8 xv[4], av[NR][4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int kk = min(k + 32 * e, s.k - 32);          // (k is a multiple of 64)
      xv[e] = *reinterpret_cast<const f16x8*>(x + kk);
#pragma unroll
      for (int i = 0; i < NR; ++i) av[i][e] = *reinterpret_cast<const f16x8*>(ar[i] + kk);
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (k + 32 * e >= end) break;
#pragma unroll
      for (int i = 0; i < NR; ++i)
        acc[i] = __builtin_amdgcn_mfma_f32_16x16x32_f16(xv[e], av[i][e], acc[i], 0, 0, 0);
    }
  }
#pragma unroll
  for (int i = 0; i < NR; ++i) red[wave][i][lane] = acc[i];
  __syncthreads();
  const float f = s.scale != nullptr ? s.scale[slot] : 1.f;
  for (int e = threadIdx.x; e < NR * 64; e += 512) {
    const int i = e >> 6, l = e & 63, r = 16 * i + (l & 15);
    f32x4 sum = red[0][i][l];
#pragma unroll
    for (int w = 1; w < 8; ++w) sum += red[w][i][l];
    if (r >= s.rp) continue;
    // D[4 (l / 16) + v][l % 16]
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const int row = 4 * (l >> 4) + v;
      if (row < rows)
        s.t[((int64_t)sp * s.m + s.plan.order[p0 + row]) * s.rp + r] = r < s.rank ? f * sum[v] : 0.f;
    }
  }
}

}  // namespace qlin
