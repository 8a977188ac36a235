// Host-side argument checks shared by the C-ABI entry points (no HIP call but
// check_device's).
#pragma once

#include <hip/hip_runtime.h>

#include <stdint.h>
#include <string.h>

#include "../../include/qlin.h"
#include "plan.h"

namespace qlin {

inline thread_local int g_last_hip_error = 0;

constexpr int kMaxN = 1 << 24;
constexpr int kMaxK = 1 << 20;
constexpr int kMaxM = 1 << 20;

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

struct Range { uintptr_t lo, hi; };
inline Range range_of(const void* p, int64_t bytes) {
  const uintptr_t a = reinterpret_cast<uintptr_t>(p);
  return Range{a, a + (uintptr_t)(bytes > 0 ? bytes : 0)};
}
inline bool overlaps(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }

// Widths with a packed-code layout, and every width of the lever (scale/zero
// precompute and the fused re-quantizing GEMV from fp16 masters): the same.
inline bool valid_bits(int bits) { return bits >= 2 && bits <= 8; }
inline bool lever_bits(int bits) { return bits >= 2 && bits <= 8; }

inline qlin_status check_nk(int32_t n, int32_t k) {
  if (n < 1 || n > kMaxN || k < kBlock || k > kMaxK || (k % kBlock) != 0) return QLIN_ERR_SHAPE;
  return QLIN_OK;
}

inline qlin_status check_group(int32_t group, int32_t k) {
  return (group == kBlock || group == k) ? QLIN_OK : QLIN_ERR_GROUP;
}

inline int64_t packed_bytes(int64_t n, int64_t k, int bits) {
  return tiles_of(n) * kTile * (k / kBlock) * 2 * bits * 4;
}
inline int64_t meta_entries(int64_t n, int64_t k, int group) {
  return tiles_of(n) * kTile * (group == k ? 1 : k / kBlock);
}

inline qlin_status hip_status(hipError_t e) {
  if (e == hipSuccess) return QLIN_OK;
  g_last_hip_error = (int)e;
  return QLIN_ERR_HIP;
}

// One check per process and device: the kernels are built for gfx950 only.
inline qlin_status check_device() {
  int dev = 0;
  hipError_t e = hipGetDevice(&dev);
  if (e != hipSuccess) { g_last_hip_error = (int)e; return QLIN_ERR_NO_DEVICE; }
  static thread_local int cached_dev = -1;
  static thread_local bool cached_ok = false;
  if (dev == cached_dev) return cached_ok ? QLIN_OK : QLIN_ERR_NO_DEVICE;
  hipDeviceProp_t prop;
  e = hipGetDeviceProperties(&prop, dev);
  if (e != hipSuccess) { g_last_hip_error = (int)e; return QLIN_ERR_NO_DEVICE; }
  cached_dev = dev;
  cached_ok = strncmp(prop.gcnArchName, "gfx950", 6) == 0;
  return cached_ok ? QLIN_OK : QLIN_ERR_NO_DEVICE;
}

inline qlin_status check_weight(const qlin_weight* w, bool allow_master, bool allow16) {
  if (w == nullptr) return QLIN_ERR_NULL;
  qlin_status st = check_nk(w->n, w->k);
  if (st != QLIN_OK) return st;
  if (w->reserved != 0) return QLIN_ERR_FORMAT;
  if (w->format == QLIN_FMT_PACKED) {
    if (!valid_bits(w->bits)) return QLIN_ERR_BITS;
    if (w->ld != 0) return QLIN_ERR_SHAPE;
  } else if (w->format == QLIN_FMT_FP16_MASTER) {
    if (!allow_master) return QLIN_ERR_FORMAT;
    if (!(lever_bits(w->bits) || (allow16 && w->bits == 16))) return QLIN_ERR_BITS;
    if (w->ld < w->k) return QLIN_ERR_SHAPE;
    if (w->ld % 8 != 0) return QLIN_ERR_ALIGN;
  } else {
    return QLIN_ERR_FORMAT;
  }
  if (w->data == nullptr) return QLIN_ERR_NULL;
  if (!aligned16(w->data)) return QLIN_ERR_ALIGN;
  if (w->bits != 16) {
    st = check_group(w->group, w->k);
    if (st != QLIN_OK) return st;
    if (w->scale == nullptr || w->zero == nullptr) return QLIN_ERR_NULL;
    if (!aligned16(w->scale) || !aligned16(w->zero)) return QLIN_ERR_ALIGN;
  }
  return QLIN_OK;
}

inline int64_t weight_bytes(const qlin_weight* w) {
  if (w->format == QLIN_FMT_PACKED) return packed_bytes(w->n, w->k, w->bits);
  return ((int64_t)(w->n - 1) * w->ld + w->k) * 2;
}

inline bool output_overlaps_weight(const qlin_weight* w, Range out) {
  if (overlaps(out, range_of(w->data, weight_bytes(w)))) return true;
  if (w->bits != 16) {
    const int64_t me = meta_entries(w->n, w->k, w->group);
    if (overlaps(out, range_of(w->scale, me * 2))) return true;
    if (overlaps(out, range_of(w->zero, me))) return true;
  }
  return false;
}

}  // namespace qlin
