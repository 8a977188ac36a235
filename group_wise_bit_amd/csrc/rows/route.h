// Routing to experts (gfx950, wave64).
#pragma once

#include "../device_common.h"

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

// The largest of the wave's (key, index) pairs, the lower index among equal
// keys; every lane returns it.
__device__ __forceinline__ void wave_best(double& key, int& idx) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) {
    const double ok = __shfl_xor(key, d);
    const int oi = __shfl_xor(idx, d);
    if (ok > key || (ok == key && oi < idx)) { key = ok; idx = oi; }
  }
}

__device__ __forceinline__ double wave_sum(double v) {
#pragma unroll
  for (int d = 32; d > 0; d >>= 1) v += __shfl_xor(v, d);
  return v;
}

// One wave per row; lane l holds experts l, l + 64, ... (EPL of them), scores
// and keys in 64 bits.  A masked expert's key is -infinity.
template <int EPL>
__global__ __launch_bounds__(kRouteWaves * 64) void k_route(const RouteArgs a) {
  constexpr double kInf = __builtin_inf();
  __shared__ double val[kRouteWaves][EPL * 64];
  const int lane = lane_id(), wave = wave_id();
  const int row = blockIdx.x * kRouteWaves + wave;
  if (row >= a.m) return;
  const float* lp = a.logits + (int64_t)row * a.ld;
  double x[EPL], p[EPL], b[EPL];
  bool live[EPL];
  double top = -kInf;
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    const int e = lane + 64 * i;
    const float l = e < a.experts ? lp[e] : -__builtin_inff();
    const float bi = a.bias != nullptr && e < a.experts ? a.bias[e] : 0.f;
    live[i] = l > -__builtin_inff();          // false for NaN
    x[i] = live[i] ? (double)fminf(l, 3.402823466e38f) : -kInf;
    b[i] = bi;
    top = fmax(top, x[i]);
  }
  if (a.sigmoid) {
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = live[i] ? 1.0 / (1.0 + exp(-x[i])) : 0.0;
  } else {
    int none = 0;
    wave_best(top, none);
    double sum = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      p[i] = live[i] ? exp(x[i] - top) : 0.0;
      sum += p[i];
    }
    sum = wave_sum(sum);
#pragma unroll
    for (int i = 0; i < EPL; ++i) p[i] = live[i] ? p[i] / sum : 0.0;
  }
  double key[EPL];
#pragma unroll
  for (int i = 0; i < EPL; ++i) {
    if (!(b[i] > -kInf)) live[i] = false;     // a bias of -inf or NaN
    b[i] = live[i] ? p[i] + b[i] : -kInf;     // the biased score
    key[i] = a.bias != nullptr ? b[i] : (live[i] ? x[i] : -kInf);
  }
  if (a.groups > 1) {
    const int per = a.experts / a.groups;
#pragma unroll
    for (int i = 0; i < EPL; ++i) val[wave][lane + 64 * i] = a.group_top == 1 ? key[i] : b[i];
    __builtin_amdgcn_wave_barrier();
    // lane g: the value of group g
    double v = -kInf;
    if (lane < a.groups) {
      double first = -kInf, second = -kInf;
      for (int j = 0; j < per; ++j) {
        const double w = val[wave][lane * per + j];
        second = fmax(second, fmin(first, w));
        first = fmax(first, w);
      }
      v = a.group_top == 1 || second == -kInf ? first : first + second;
    }
    uint64_t kept = 0;
    for (int j = 0; j < a.top_groups; ++j) {
      double best = v;
      int g = v == -kInf ? 64 : lane;
      wave_best(best, g);
      if (g >= 64) break;
      kept |= 1ull << g;
      if (lane == g) v = -kInf;
    }
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int e = lane + 64 * i;
      if (e >= a.experts || !((kept >> (e / per)) & 1)) key[i] = -kInf;
    }
  }
  // the best top_k, one after the other; lane j keeps the j-th
  int my_id = -1;
  double my_p = 0.0;
  for (int j = 0; j < a.top_k; ++j) {
    double best = -kInf;
    int at = 1 << 20;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (key[i] > best) { best = key[i]; at = lane + 64 * i; }
    wave_best(best, at);
    if (best == -kInf) break;
    double ps = 0.0;
#pragma unroll
    for (int i = 0; i < EPL; ++i)
      if (at == lane + 64 * i) {
        ps = p[i];
        key[i] = -kInf;
      }
    ps = __shfl(ps, at & 63);
    if (lane == j) { my_id = at; my_p = ps; }
  }
  if (a.renormalize) {
    const double sum = wave_sum(my_p);
    my_p = sum > 0.0 ? my_p / sum : 0.0;
  }
  if (lane < a.top_k) {
    const int64_t o = (int64_t)row * a.top_k + lane;
    a.ids[o] = my_id;
    a.weights[o] = (float)(my_p * (double)a.scale);
  }
}

}  // namespace qlin
