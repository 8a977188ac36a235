// Entry point of qlin_sample.h: host checks, launches.
#include <hip/hip_runtime.h>

#include "../../../include/qlin_sample.h"
#include "../checks.h"
#include "sample.h"

using namespace qlin;

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int kMaxVocab = 1 << 18;

}  // namespace

extern "C" {

int64_t qlin_sample_workspace_bytes(int32_t m, int32_t vocab) {
  if (m < 1 || m > kMaxM || vocab < 1 || vocab > kMaxVocab) return 0;
  return kCounterBytes;
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
  hipLaunchKernelGGL(k_sample_row, dim3(m), dim3(kSampleThreads), 0, stream, a);
  return hip_status(hipGetLastError());
}

}  // extern "C"
