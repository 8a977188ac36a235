// The cache's kernels for one pair of widths, compiled as its own object with
// -DQLIN_INST_KB=<keys' bits> -DQLIN_INST_VB=<values' bits>, and
// -DQLIN_INST_PART=0 for stores and reads, 1 for attention.
#include "kv_plan.h"

namespace qlin {

#if QLIN_INST_PART == 0
template <int KB, int VB>
void launch_kv_store(const KvStoreArgs& a, int d, dim3 grid, hipStream_t st) {
  if (d == 64) hipLaunchKernelGGL((k_kv_store<64, KB, VB>), grid, dim3(256), 0, st, a);
  else if (d == 128) hipLaunchKernelGGL((k_kv_store<128, KB, VB>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((k_kv_store<256, KB, VB>), grid, dim3(256), 0, st, a);
}

template <int D, int KB, int VB>
void launch_read_dim(const KvReadArgs& a, bool wide, dim3 grid, hipStream_t st) {
  if (wide) hipLaunchKernelGGL((k_kv_read<D, KB, VB, true>), grid, dim3(256), 0, st, a);
  else hipLaunchKernelGGL((k_kv_read<D, KB, VB, false>), grid, dim3(256), 0, st, a);
}

template <int KB, int VB>
void launch_kv_read(const KvReadArgs& a, int d, bool wide, dim3 grid, hipStream_t st) {
  if (d == 64) launch_read_dim<64, KB, VB>(a, wide, grid, st);
  else if (d == 128) launch_read_dim<128, KB, VB>(a, wide, grid, st);
  else launch_read_dim<256, KB, VB>(a, wide, grid, st);
}

template void launch_kv_store<QLIN_INST_KB, QLIN_INST_VB>(const KvStoreArgs&, int, dim3, hipStream_t);
template void launch_kv_read<QLIN_INST_KB, QLIN_INST_VB>(const KvReadArgs&, int, bool, dim3,
                                                         hipStream_t);
#else
template <int D, int KB, int VB>
void launch_attend_dim(const AttendArgs& a, hipStream_t st) {
  const int groups = a.whole ? a.s.seqs * a.kv_heads * a.rts : a.groups;
  hipLaunchKernelGGL((k_attend<D, KB, VB>), dim3(groups), dim3(256), 0, st, a);
  if (!a.whole) hipLaunchKernelGGL((k_attend_join<D>), dim3(a.s.seqs, a.heads), dim3(256), 0, st, a);
}

template <int KB, int VB>
void launch_attend(const AttendArgs& a, int d, hipStream_t st) {
  if (d == 64) launch_attend_dim<64, KB, VB>(a, st);
  else if (d == 128) launch_attend_dim<128, KB, VB>(a, st);
  else launch_attend_dim<256, KB, VB>(a, st);
}

template void launch_attend<QLIN_INST_KB, QLIN_INST_VB>(const AttendArgs&, int, hipStream_t);
#endif

}  // namespace qlin
