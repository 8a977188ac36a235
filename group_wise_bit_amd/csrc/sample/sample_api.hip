// Entry point of qlin_sample.h: host checks, launches.
#include <hip/hip_runtime.h>

#include "../../../include/qlin_sample.h"
#include "../checks.h"
#include "split.h"

using namespace qlin;

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int kMaxVocab = kSlice * kSlices;

int64_t align256(int64_t b) { return (b + 255) & ~(int64_t)255; }

// Rows are drawn in batches of at most kBatchRows rows and kBatchSlices slices, so that the
// workspace is bounded (below 72 MB): enough of them to fill the chip several times over.
constexpr int kBatchSlices = 8192;
constexpr int kBatchRows = 512;

struct SamplePlan {
  int slices, rows;
  int64_t mass, count, stat, plan, list, bytes;    // offsets in the workspace, and its size
};

SamplePlan sample_plan(int m, int vocab) {
  SamplePlan p{};
  p.slices = (vocab + kSlice - 1) / kSlice;
  const int most = kBatchSlices / p.slices < kBatchRows ? kBatchSlices / p.slices : kBatchRows;
  p.rows = m < most ? m : most;
  const int64_t items = (int64_t)p.rows * p.slices;
  p.mass = kCounterBytes;
  p.count = align256(p.mass + items * kSums * (int64_t)sizeof(double));
  p.stat = align256(p.count + items * kSums * (int64_t)sizeof(uint32_t));
  p.plan = align256(p.stat + items * (int64_t)sizeof(SliceStat));
  p.list = align256(p.plan + p.rows * (int64_t)sizeof(RowPlanS));
  p.bytes = p.list + p.rows * (int64_t)kListMax * (int64_t)sizeof(uint2);
  return p;
}

}  // namespace

extern "C" {

int64_t qlin_sample_workspace_bytes(int32_t m, int32_t vocab) {
  if (m < 1 || m > kMaxM || vocab < 1 || vocab > kMaxVocab) return 0;
  return sample_plan(m, vocab).bytes;
}

qlin_status qlin_sample(const qlin_sampling* s, const float* logits, int32_t m, int32_t vocab,
                        int64_t ld, const float* u, int32_t* ids, float* probs, void* workspace,
                        int64_t workspace_bytes, hipStream_t stream) {
  if (s == nullptr) return QLIN_ERR_NULL;
  if (m < 0 || m > kMaxM || vocab < 1 || vocab > kMaxVocab || ld < vocab) return QLIN_ERR_SHAPE;
  if (m == 0) return QLIN_OK;
  if (logits == nullptr || u == nullptr || ids == nullptr) return QLIN_ERR_NULL;
  if (!aligned4(logits) || !aligned4(u) || !aligned4(ids) || !aligned4(probs) ||
      !aligned4(s->temperature) || !aligned4(s->top_k) || !aligned4(s->top_p) ||
      !aligned4(s->min_p) || !aligned16(workspace))
    return QLIN_ERR_ALIGN;
  if (workspace == nullptr || workspace_bytes < qlin_sample_workspace_bytes(m, vocab))
    return QLIN_ERR_WORKSPACE;
  const int64_t vec = (int64_t)m * 4;
  const Range out[3] = {range_of(workspace, workspace_bytes), range_of(ids, vec),
                        range_of(probs, probs != nullptr ? vec : 0)};
  const Range in[6] = {range_of(logits, ((int64_t)(m - 1) * ld + vocab) * 4), range_of(u, vec),
                       range_of(s->temperature, s->temperature != nullptr ? vec : 0),
                       range_of(s->top_k, s->top_k != nullptr ? vec : 0),
                       range_of(s->top_p, s->top_p != nullptr ? vec : 0),
                       range_of(s->min_p, s->min_p != nullptr ? vec : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i], r)) return QLIN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return QLIN_ERR_ALIAS;
  }
  const qlin_status st = check_device();
  if (st != QLIN_OK) return st;
  SampleArgs a{};
  a.temperature = s->temperature;
  a.top_k = s->top_k;
  a.top_p = s->top_p;
  a.min_p = s->min_p;
  a.logits = logits;
  a.u = u;
  a.ld = ld;
  a.ids = ids;
  a.probs = probs;
  a.m = m;
  a.vocab = vocab;
  const SamplePlan p = sample_plan(m, vocab);
  char* const base = static_cast<char*>(workspace);
  SplitArgs b{};
  b.s = a;
  b.slices = p.slices;
  b.cum_mass = reinterpret_cast<double*>(base + p.mass);
  b.cum_count = reinterpret_cast<uint32_t*>(base + p.count);
  b.stat = reinterpret_cast<SliceStat*>(base + p.stat);
  b.plan = reinterpret_cast<RowPlanS*>(base + p.plan);
  b.list = reinterpret_cast<uint2*>(base + p.list);
  const bool cuts = a.top_k != nullptr || a.top_p != nullptr || a.min_p != nullptr;
  for (b.row0 = 0; b.row0 < m; b.row0 += p.rows) {
    const int rows = m - b.row0 < p.rows ? m - b.row0 : p.rows;
    hipLaunchKernelGGL(k_sample_bins, dim3(rows * p.slices), dim3(kBinThreads), 0, stream, b);
    hipLaunchKernelGGL(k_sample_bounds, dim3(rows), dim3(kBins), 0, stream, b);
    if (cuts)
      hipLaunchKernelGGL(k_sample_gather, dim3(rows * p.slices), dim3(kBinThreads), 0, stream, b);
    hipLaunchKernelGGL(k_sample_pick, dim3(rows), dim3(kPickThreads), 0, stream, b);
  }
  return hip_status(hipGetLastError());
}

}  // extern "C"
