// Launchers of the cache's kernels, one object per pair of widths (kv_inst.hip).
#pragma once

#include "attend.h"
#include "kv_store.h"

namespace qlin {

// Work-groups of the attention: as many as the launch bounds let 256 CUs hold at once (or fewer),
// so that none waits for another's end.
inline int attend_groups(int d, int kb, int vb) {
  return 256 * attend_occupancy(d, kb, vb);
}

template <int KB, int VB>
void launch_kv_store(const KvStoreArgs& a, int d, dim3 grid, hipStream_t st);
template <int KB, int VB>
void launch_kv_read(const KvReadArgs& a, int d, bool wide, dim3 grid, hipStream_t st);
template <int KB, int VB>
void launch_attend(const AttendArgs& a, int d, hipStream_t st);

}  // namespace qlin
