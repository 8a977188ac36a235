// The cache tile and what its kernels share (gfx950, wave64).
#pragma once

#include "../device_common.h"

namespace qlin {

constexpr int kKvTile = 32;      // tokens of a cache tile

// Byte offsets in a tile of D-dim heads with KB and VB bits.
template <int D, int KB, int VB>
struct KvTile {
  static constexpr int G = D / 64;
  static constexpr int k = 0;
  static constexpr int v = k + 4 * D * KB;
  static constexpr int ks = v + 4 * D * VB;
  static constexpr int vs = ks + (KB < 16 ? 64 * G : 0);
  static constexpr int kz = vs + (VB < 16 ? 64 * G : 0);
  static constexpr int vz = kz + (KB < 16 ? 32 * G : 0);
  static constexpr int bytes = vz + (VB < 16 ? 32 * G : 0);
};

constexpr int kv_tile_bytes(int d, int kb, int vb) {
  return 4 * d * (kb + vb) + ((kb < 16) + (vb < 16)) * 96 * (d / 64);
}

// The sequences of a call.
struct KvSeqs {
  const int32_t* table;
  const int32_t* lengths;
  const int32_t* starts;     // (rows of a store or read) NULL: one row each
  int64_t ld;
  int seqs, width, pages;
  int m;                     // rows of the call
  int page_log;              // log2 of the tiles of a page
};

typedef uint32_t u32x2 __attribute__((ext_vector_type(2)));

// The larger ones of two pairs of fp16 numbers (of a NaN and another the other one).
__device__ __forceinline__ uint32_t pk_max(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("v_pk_max_f16 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
  return r;
}

// Inclusive sum over the wave's lanes (within rows of 16, then row 0's into row 1
// and 2's into 3, then the lower half's into the upper).
template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int v) {
  return v + __builtin_amdgcn_update_dpp(0, v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ int scan64(int v) {
  v = dpp_add<0x111, 0xF>(v);
  v = dpp_add<0x112, 0xF>(v);
  v = dpp_add<0x114, 0xF>(v);
  v = dpp_add<0x118, 0xF>(v);
  v = dpp_add<0x142, 0xA>(v);
  return dpp_add<0x143, 0xC>(v);
}

}  // namespace qlin
