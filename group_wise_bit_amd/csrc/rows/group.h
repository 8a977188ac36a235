// Kernels beside the row-wise products that no bit width changes: grouping rows
// by expert, the sum over a token's experts, the adapters' first product.
#pragma once

#include "rows.h"

namespace qlin {

// ------------------------------------------------------------ grouping rows --
// A stable counting sort of `count` ids: positions 0 .. count-1 hold the
// indexes of the ids, bucket after bucket, in order within a bucket; ids
// outside [0, buckets) share a last bucket.  Also the table of row tiles: up
// to `rows` positions of one bucket each.  One work-group: wave w takes the
// w-th 16th of the ids, counts it (lanes with equal ids find each other by
// ballots over the id's bits, their first lane adds to the wave's own
// counters), the counters are turned into starts, and a second pass writes
// the positions.  No atomics: the order is the ids' own.
constexpr int kPlanWaves = 16;

// Lanes of the wave (in `live`) whose id equals this lane's; nbits covers the ids.
__device__ __forceinline__ uint64_t same_id(int id, uint64_t live, int nbits) {
  uint64_t m = live;
  for (int b = 0; b < nbits; ++b) {
    const uint64_t one = __builtin_amdgcn_ballot_w64((id >> b) & 1);
    m &= ((id >> b) & 1) ? one : ~one;
  }
  return m;
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

__global__ __launch_bounds__(kPlanWaves * 64) void k_rows_plan(
    const int32_t* __restrict__ ids, int count, int buckets, int rows, RowPlan plan) {
  __shared__ int hist[kPlanWaves][kMaxExperts + 1];
  __shared__ int part[kPlanWaves][2];
  const int tid = threadIdx.x, lane = lane_id(), wave = wave_id();
  for (int i = tid; i < kPlanWaves * (kMaxExperts + 1); i += kPlanWaves * 64) (&hist[0][0])[i] = 0;
  __syncthreads();
  const int nbits = 32 - __builtin_clz(buckets);
  const int share = ((count + kPlanWaves * 64 - 1) / (kPlanWaves * 64)) * 64;
  const int i0 = min(count, wave * share), i1 = min(count, i0 + share);
  auto bucket_of = [&](int i) __attribute__((always_inline)) {
    const int id = i < i1 ? ids[i] : 0;
    return (uint32_t)id < (uint32_t)buckets ? id : buckets;
  };
  for (int b = i0; b < i1; b += 64) {
    const int id = bucket_of(b + lane);
    const uint64_t live = __builtin_amdgcn_ballot_w64(b + lane < i1);
    const uint64_t m = same_id(id, live, nbits);
    if (b + lane < i1 && (m & ((1ull << lane) - 1)) == 0) hist[wave][id] += __builtin_popcountll(m);
    counters_written();
  }
  __syncthreads();
  // thread t: bucket t's count, starts of its waves, its start and its tiles'
  int total = 0;
  if (tid <= buckets) {
    for (int w = 0; w < kPlanWaves; ++w) {
      const int c = hist[w][tid];
      hist[w][tid] = total;
      total += c;
    }
  }
  const int mine = tid < buckets ? (total + rows - 1) / rows : 0;
  int end = total, tend = mine;
  group_scan2(end, tend, part);
  const int start = end - total;
  if (tid <= buckets) {
    for (int w = 0; w < kPlanWaves; ++w) hist[w][tid] += start;
    plan.offs[tid] = start;
    if (tid == buckets) {
      plan.offs[buckets + 1] = end;
      *plan.ntiles = tend;
    }
    for (int i = 0; i < mine; ++i) {
      plan.tiles[2 * (tend - mine + i)] = tid;
      plan.tiles[2 * (tend - mine + i) + 1] = start + i * rows;
    }
  }
  __syncthreads();
  for (int b = i0; b < i1; b += 64) {
    const int id = bucket_of(b + lane);
    const uint64_t live = __builtin_amdgcn_ballot_w64(b + lane < i1);
    const uint64_t m = same_id(id, live, nbits);
    const int before = __builtin_popcountll(m & ((1ull << lane) - 1));
    int at = 0;
    if (b + lane < i1) {
      at = hist[wave][id] + before;
      plan.order[at] = b + lane;
    }
    counters_written();
    if (b + lane < i1 && before == 0) hist[wave][id] = at + __builtin_popcountll(m);
    counters_written();
  }
}

// ------------------------------------------------- sum over a token's experts --
// Y[i, :] = the rows of its valid (token, slot) pairs, added in slot order.
// One thread: 4 columns of one token (n is a multiple of 64).
__global__ __launch_bounds__(256) void k_rows_combine(
    const float* __restrict__ d, const int32_t* __restrict__ ids, int m, int top_k, int experts,
    int n, float* __restrict__ y, uint16_t* __restrict__ y16, int64_t ldy) {
  const int n4 = n / 4;
  for (int64_t q = (int64_t)blockIdx.x * 256 + threadIdx.x; q < (int64_t)m * n4;
       q += (int64_t)gridDim.x * 256) {
    const int64_t i = q / n4;
    const int c = (int)(q % n4) * 4;
    f32x4 s = {0.f, 0.f, 0.f, 0.f};
    for (int j = 0; j < top_k; ++j)
      if ((uint32_t)ids[i * top_k + j] < (uint32_t)experts)
        s += *reinterpret_cast<const f32x4*>(d + (i * top_k + j) * n + c);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      if (y != nullptr) y[i * ldy + c + e] = s[e];
      if (y16 != nullptr) y16[i * ldy + c + e] = __builtin_bit_cast(uint16_t, (f16)s[e]);
    }
  }
}

// ------------------------------------------------------ A x of the adapters --
// t = scale * A x of one row, kept as a power of two 2^e and the fp16 halves
// of t 2^-e (high, then what is left of it), |t 2^-e| < 2^15: 22 bits of the
// row's largest entry, for any finite t.
__device__ __forceinline__ float half_scale(float largest) {
  if (!(largest > 0.f) || largest > 3.402823466e38f) return 1.f;
  const int e = ((__builtin_bit_cast(uint32_t, largest) >> 23) & 255) - 127;   // floor(log2)
  const int s = max(-126, min(127, e - 14));
  return __builtin_bit_cast(float, (uint32_t)(s + 127) << 23);
}
__device__ __forceinline__ void store_halves(uint16_t* hi, uint16_t* lo, float t) {
  const f16 a = (f16)t;
  const float rest = t - (float)a;
  const f16 b = (f16)(__builtin_isfinite(rest) ? rest : 0.f);
  *hi = __builtin_bit_cast(uint16_t, a);
  *lo = __builtin_bit_cast(uint16_t, b);
}

struct ShrinkArgs {
  const uint16_t* X;
  int64_t ldx;
  int m, k, slots, rank, rp;
  const int32_t* ids;
  const uint16_t* a;      // [slots][rank][k]
  const float* scale;     // [slots] or null
  uint16_t* t;            // [m][2][rp]
  float* tscale;          // [m]
};

// One work-group per row: its waves take the rank rows w, w + 4, ...
__global__ __launch_bounds__(256) void k_lora_shrink_row(const ShrinkArgs s) {
  __shared__ float red[128];
  const int lane = lane_id(), wave = wave_id();
  const int64_t row = blockIdx.x;
  const int slot = s.ids[row];
  if ((uint32_t)slot >= (uint32_t)s.slots) return;
  const uint16_t* x = s.X + row * s.ldx;
  for (int r = wave; r < s.rank; r += 4) {
    const uint16_t* ar = s.a + ((int64_t)slot * s.rank + r) * s.k;
    float sum = 0.f;
    for (int k = 8 * lane; k < s.k; k += 512) {
      const uint4 av = *reinterpret_cast<const uint4*>(ar + k);
      const uint4 xv = *reinterpret_cast<const uint4*>(x + k);
      sum = __builtin_amdgcn_fdot2(as_h2(av.x), as_h2(xv.x), sum, false);
      sum = __builtin_amdgcn_fdot2(as_h2(av.y), as_h2(xv.y), sum, false);
      sum = __builtin_amdgcn_fdot2(as_h2(av.z), as_h2(xv.z), sum, false);
      sum = __builtin_amdgcn_fdot2(as_h2(av.w), as_h2(xv.w), sum, false);
    }
    sum = row_sum16(sum);
    sum += __shfl_xor(sum, 16);
    sum += __shfl_xor(sum, 32);
    if (lane == 0) red[r] = sum;
  }
  __syncthreads();
  if (wave != 0) return;
  const float f = s.scale != nullptr ? s.scale[slot] : 1.f;
  const float t0 = lane < s.rank ? f * red[lane] : 0.f;
  const float t1 = lane + 64 < s.rank ? f * red[lane + 64] : 0.f;
  float top = fmaxf(__builtin_fabsf(t0), __builtin_fabsf(t1));
#pragma unroll
  for (int d = 1; d < 64; d *= 2) top = fmaxf(top, __shfl_xor(top, d));
  const float p = half_scale(top);
  uint16_t* out = s.t + row * 2 * s.rp;
  const float inv = 1.f / p;
  if (lane < s.rp) store_halves(out + lane, out + s.rp + lane, t0 * inv);
  if (lane + 64 < s.rp) store_halves(out + lane + 64, out + s.rp + lane + 64, t1 * inv);
  if (lane == 0) s.tscale[row] = p;
}

}  // namespace qlin
