// Entry points of qlin_kv.h: host checks, workspace layout, launches.
#include <hip/hip_runtime.h>

#include <math.h>

#include "../../../include/qlin_kv.h"
#include "../checks.h"
#include "kv_plan.h"

using namespace qlin;

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int kMaxSeqs = 1 << 16;
constexpr int kMaxKvHeads = 256;
constexpr int kMaxHeads = 1024;
constexpr int64_t kMaxRoom = 1 << 27;      // tokens of a table row
constexpr float kMaxScale = 1 << 20;

bool kv_dim(int d) { return d == 64 || d == 128 || d == 256; }
bool kv_page_size(int p) { return p == 32 || p == 64 || p == 128 || p == 256; }
bool kv_bits(int b) { return b == 4 || b == 8 || b == 16; }

int64_t page_bytes(const qlin_kv_cache* c) {
  return (int64_t)(c->page / kKvTile) * kv_tile_bytes(c->head_dim, c->k_bits, c->v_bits);
}
Range cache_range(const qlin_kv_cache* c) {
  return range_of(c->data, (int64_t)c->pages * c->kv_heads * page_bytes(c));
}

// Sizes only.
qlin_status check_sizes(const qlin_kv_cache* c, const qlin_kv_seqs* s) {
  if (c == nullptr || s == nullptr) return QLIN_ERR_NULL;
  if (!kv_bits(c->k_bits) || !kv_bits(c->v_bits)) return QLIN_ERR_BITS;
  if (c->pages < 1 || c->kv_heads < 1 || c->kv_heads > kMaxKvHeads || !kv_dim(c->head_dim) ||
      !kv_page_size(c->page))
    return QLIN_ERR_SHAPE;
  if (s->seqs < 0 || s->seqs > kMaxSeqs || s->width < 1 ||
      (int64_t)s->width * c->page > kMaxRoom || s->ld < s->width)
    return QLIN_ERR_SHAPE;
  return QLIN_OK;
}

qlin_status check_pointers(const qlin_kv_cache* c, const qlin_kv_seqs* s) {
  if (c->data == nullptr || s->table == nullptr || s->lengths == nullptr) return QLIN_ERR_NULL;
  if (!aligned16(c->data) || !aligned4(s->table) || !aligned4(s->lengths)) return QLIN_ERR_ALIGN;
  return QLIN_OK;
}

// Whether an output overlaps the tables of the sequences.
bool overlaps_seqs(const qlin_kv_seqs* s, const int32_t* starts, Range r) {
  return overlaps(r, range_of(s->table, ((int64_t)(s->seqs - 1) * s->ld + s->width) * 4)) ||
         overlaps(r, range_of(s->lengths, (int64_t)s->seqs * 4)) ||
         overlaps(r, range_of(starts, starts != nullptr ? (int64_t)(s->seqs + 1) * 4 : 0));
}

// Whether rows of `bytes` at a and at b, both `pitch` bytes apart, take turns (the
// columns of one wider matrix).
bool rows_apart(const void* a, const void* b, int64_t pitch, int64_t bytes) {
  if (pitch == 0) return false;
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  const int64_t apart = (int64_t)((x > y ? x - y : y - x) % (uintptr_t)pitch);
  return apart >= bytes && pitch - apart >= bytes;
}

KvSeqs make_seqs(const qlin_kv_cache* c, const qlin_kv_seqs* s, const int32_t* starts, int m) {
  KvSeqs k{};
  k.table = s->table;
  k.lengths = s->lengths;
  k.starts = starts;
  k.ld = s->ld;
  k.seqs = s->seqs;
  k.width = s->width;
  k.pages = c->pages;
  k.m = m;
  for (int t = c->page / kKvTile; t > 1; t /= 2) ++k.page_log;
  return k;
}

// (tile, head and part) of a store or read: a sequence's rows begin and end
// within tiles, so m rows of seqs sequences touch m / 32 + 2 seqs at most.
dim3 rows_grid(const qlin_kv_cache* c, const qlin_kv_seqs* s, const int32_t* starts, int m) {
  const int n = s->seqs < m ? s->seqs : m;
  const int items = starts == nullptr ? s->seqs : m / kKvTile + 2 * n;
  return dim3(items, (c->kv_heads * (2 + c->head_dim / 64) + 3) / 4);
}
bool grid_fits(dim3 g, int threads) { return (int64_t)g.x * g.y * threads < ((int64_t)1 << 32); }

template <template <int, int> class F, typename... A>
void by_bits(const qlin_kv_cache* c, A&&... a) {
  switch (c->k_bits * 32 + c->v_bits) {
    case 4 * 32 + 4: F<4, 4>::run(a...); break;
    case 4 * 32 + 8: F<4, 8>::run(a...); break;
    case 4 * 32 + 16: F<4, 16>::run(a...); break;
    case 8 * 32 + 4: F<8, 4>::run(a...); break;
    case 8 * 32 + 8: F<8, 8>::run(a...); break;
    case 8 * 32 + 16: F<8, 16>::run(a...); break;
    case 16 * 32 + 4: F<16, 4>::run(a...); break;
    case 16 * 32 + 8: F<16, 8>::run(a...); break;
    default: F<16, 16>::run(a...); break;
  }
}
template <int KB, int VB>
struct Store {
  static void run(const KvStoreArgs& a, int d, dim3 g, hipStream_t st) {
    launch_kv_store<KB, VB>(a, d, g, st);
  }
};
template <int KB, int VB>
struct Read {
  static void run(const KvReadArgs& a, int d, bool wide, dim3 g, hipStream_t st) {
    launch_kv_read<KB, VB>(a, d, wide, g, st);
  }
};
template <int KB, int VB>
struct Attend {
  static void run(const AttendArgs& a, int d, hipStream_t st) { launch_attend<KB, VB>(a, d, st); }
};

// Sequences of tables up to this length are not split: a work-group has all of one, and
// nothing is joined.  Kernel times unsplit : split (its join, 4.0 to 5.5 us and a launch, apart), in us.
// One sequence, 64 dims of 8 bits: 300 tokens 6.1 : 5.4, 1024 8.8 : 5.4, 2048 13.8 : 5.5; 128
// dims of 4 bits: 512 9.6 : 6.7, 1024 13.3 : 8.0, 2048 20.3 : 6.8; 256 dims of 16 bits: 1024 20.4 :
// 10.0.  48 ragged ones, 128 dims of 4 bits: up to 300 9.7 : 11.3, 1024 16.7 : 14.1, 2048 25.0 : 19.9.
// So the limit is where 64 and 128 dims of up to 8 bits come out even, join and launch counted; wider
// tiles do so at fewer tokens (256 dims of 16 bits at 1024 lose 5 us by it), and a short
// sequence under a long table is split.
constexpr int64_t kWholeTokens = 1024;

struct AttendPlan {
  int rows, rts, groups;
  int64_t part, stat, bytes;     // offsets in the workspace, and its size
};

AttendPlan attend_plan(const qlin_kv_cache* c, const qlin_kv_seqs* s, int heads) {
  AttendPlan p{};
  const int ratio = heads / c->kv_heads;
  p.rows = ratio < kAttendRows ? ratio : kAttendRows;
  p.rts = (ratio + kAttendRows - 1) / kAttendRows;
  const int64_t most = (int64_t)s->seqs * c->kv_heads * p.rts *
                       ((int64_t)s->width * (c->page / kKvTile));
  const int64_t groups = (most + kAttendWaves - 1) / kAttendWaves;
  const int most_groups = attend_groups(c->head_dim, c->k_bits, c->v_bits);
  p.groups = (int)(groups < most_groups ? groups : most_groups);
  p.part = kCounterBytes;
  p.stat = p.part + 2 * (int64_t)p.groups * p.rows * c->head_dim * 4;
  p.bytes = p.stat + 2 * (int64_t)p.groups * p.rows * 2 * 4;
  return p;
}

qlin_status check_heads(const qlin_kv_cache* c, int32_t heads) {
  return heads < 1 || heads > kMaxHeads || heads % c->kv_heads != 0 ? QLIN_ERR_SHAPE : QLIN_OK;
}

}  // namespace

extern "C" {

int64_t qlin_kv_page_bytes(int32_t head_dim, int32_t page, int32_t k_bits, int32_t v_bits) {
  if (!kv_dim(head_dim) || !kv_page_size(page) || !kv_bits(k_bits) || !kv_bits(v_bits)) return 0;
  return (int64_t)(page / kKvTile) * kv_tile_bytes(head_dim, k_bits, v_bits);
}

qlin_status qlin_kv_write(const qlin_kv_cache* cache, const uint16_t* K, int64_t ld_k,
                          const uint16_t* V, int64_t ld_v, int32_t m, const qlin_kv_seqs* seqs,
                          const int32_t* starts, hipStream_t stream) {
  qlin_status st = check_sizes(cache, seqs);
  if (st != QLIN_OK) return st;
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (m < 0 || m > kMaxM || ld_k < row || ld_v < row) return QLIN_ERR_SHAPE;
  if (ld_k % 8 != 0 || ld_v % 8 != 0) return QLIN_ERR_ALIGN;
  if (m == 0 || seqs->seqs == 0) return QLIN_OK;
  if (starts == nullptr && m < seqs->seqs) return QLIN_ERR_SHAPE;
  st = check_pointers(cache, seqs);
  if (st != QLIN_OK) return st;
  if (K == nullptr || V == nullptr) return QLIN_ERR_NULL;
  if (!aligned16(K) || !aligned16(V) || !aligned4(starts)) return QLIN_ERR_ALIGN;
  const Range out = cache_range(cache);
  if (overlaps(out, range_of(K, ((int64_t)(m - 1) * ld_k + row) * 2)) ||
      overlaps(out, range_of(V, ((int64_t)(m - 1) * ld_v + row) * 2)) ||
      overlaps_seqs(seqs, starts, out))
    return QLIN_ERR_ALIAS;
  const dim3 grid = rows_grid(cache, seqs, starts, m);
  if (!grid_fits(grid, 256)) return QLIN_ERR_SHAPE;
  st = check_device();
  if (st != QLIN_OK) return st;
  KvStoreArgs a{};
  a.s = make_seqs(cache, seqs, starts, m);
  a.data = static_cast<uint8_t*>(cache->data);
  a.x[0] = reinterpret_cast<const f16*>(K);
  a.x[1] = reinterpret_cast<const f16*>(V);
  a.ldx[0] = ld_k;
  a.ldx[1] = ld_v;
  a.head_bytes = page_bytes(cache);
  a.kv_heads = cache->kv_heads;
  by_bits<Store>(cache, a, cache->head_dim, grid, stream);
  return hip_status(hipGetLastError());
}

qlin_status qlin_kv_read(const qlin_kv_cache* cache, const qlin_kv_seqs* seqs,
                         const int32_t* starts, int32_t m, void* K, int64_t ld_k, void* V,
                         int64_t ld_v, int32_t wide, hipStream_t stream) {
  qlin_status st = check_sizes(cache, seqs);
  if (st != QLIN_OK) return st;
  const int64_t row = (int64_t)cache->kv_heads * cache->head_dim;
  if (wide != 0 && wide != 1) return QLIN_ERR_FORMAT;
  if (m < 0 || m > kMaxM || ld_k < row || ld_v < row) return QLIN_ERR_SHAPE;
  if (ld_k % 8 != 0 || ld_v % 8 != 0) return QLIN_ERR_ALIGN;
  if (m == 0 || seqs->seqs == 0) return QLIN_OK;
  if (starts == nullptr && m < seqs->seqs) return QLIN_ERR_SHAPE;
  st = check_pointers(cache, seqs);
  if (st != QLIN_OK) return st;
  if (K == nullptr || V == nullptr) return QLIN_ERR_NULL;
  if (!aligned16(K) || !aligned16(V) || !aligned4(starts)) return QLIN_ERR_ALIGN;
  const int size = wide ? 4 : 2;
  const Range out[2] = {range_of(K, ((int64_t)(m - 1) * ld_k + row) * size),
                        range_of(V, ((int64_t)(m - 1) * ld_v + row) * size)};
  for (const Range& o : out)
    if (overlaps(o, cache_range(cache)) || overlaps_seqs(seqs, starts, o)) return QLIN_ERR_ALIAS;
  if (overlaps(out[0], out[1]) && !rows_apart(K, V, ld_k == ld_v ? ld_k * size : 0, row * size))
    return QLIN_ERR_ALIAS;
  const dim3 grid = rows_grid(cache, seqs, starts, m);
  if (!grid_fits(grid, 256)) return QLIN_ERR_SHAPE;
  st = check_device();
  if (st != QLIN_OK) return st;
  KvReadArgs a{};
  a.s = make_seqs(cache, seqs, starts, m);
  a.data = static_cast<const uint8_t*>(cache->data);
  a.x[0] = K;
  a.x[1] = V;
  a.ldx[0] = ld_k;
  a.ldx[1] = ld_v;
  a.head_bytes = page_bytes(cache);
  a.kv_heads = cache->kv_heads;
  by_bits<Read>(cache, a, cache->head_dim, wide != 0, grid, stream);
  return hip_status(hipGetLastError());
}

int64_t qlin_kv_attention_workspace_bytes(const qlin_kv_cache* cache, const qlin_kv_seqs* seqs,
                                          int32_t heads) {
  if (check_sizes(cache, seqs) != QLIN_OK || check_heads(cache, heads) != QLIN_OK ||
      seqs->seqs == 0)
    return 0;
  return attend_plan(cache, seqs, heads).bytes;
}

qlin_status qlin_kv_attention(const qlin_kv_cache* cache, const qlin_kv_seqs* seqs,
                              const uint16_t* Q, int64_t ld_q, int32_t heads, float scale,
                              int32_t window, float* O, uint16_t* O16, int64_t ld_o, float* lse,
                              void* workspace, int64_t workspace_bytes, hipStream_t stream) {
  qlin_status st = check_sizes(cache, seqs);
  if (st != QLIN_OK) return st;
  st = check_heads(cache, heads);
  if (st != QLIN_OK) return st;
  const int64_t row = (int64_t)heads * cache->head_dim;
  if (ld_q < row || ld_o < row || window < 0) return QLIN_ERR_SHAPE;
  if (!(fabsf(scale) <= kMaxScale)) return QLIN_ERR_FORMAT;
  if (ld_q % 8 != 0 || ld_o % 8 != 0) return QLIN_ERR_ALIGN;
  if (seqs->seqs == 0) return QLIN_OK;
  st = check_pointers(cache, seqs);
  if (st != QLIN_OK) return st;
  if (Q == nullptr || (O == nullptr && O16 == nullptr)) return QLIN_ERR_NULL;
  if (!aligned16(Q) || !aligned16(O) || !aligned16(O16) || !aligned4(lse) ||
      !aligned16(workspace))
    return QLIN_ERR_ALIGN;
  const AttendPlan p = attend_plan(cache, seqs, heads);
  if (!grid_fits(dim3(seqs->seqs, heads), 256)) return QLIN_ERR_SHAPE;
  if (workspace == nullptr || workspace_bytes < p.bytes) return QLIN_ERR_WORKSPACE;
  const int64_t n = seqs->seqs, span = (n - 1) * ld_o + row;
  const Range out[4] = {range_of(workspace, workspace_bytes),
                        range_of(O, O != nullptr ? span * 4 : 0),
                        range_of(O16, O16 != nullptr ? span * 2 : 0),
                        range_of(lse, lse != nullptr ? n * heads * 4 : 0)};
  for (int i = 0; i < 4; ++i) {
    if (overlaps(out[i], range_of(Q, ((n - 1) * ld_q + row) * 2)) ||
        overlaps(out[i], cache_range(cache)) || overlaps_seqs(seqs, nullptr, out[i]))
      return QLIN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return QLIN_ERR_ALIAS;
  }
  st = check_device();
  if (st != QLIN_OK) return st;
  AttendArgs a{};
  a.s = make_seqs(cache, seqs, nullptr, seqs->seqs);
  a.data = static_cast<const uint8_t*>(cache->data);
  a.head_bytes = page_bytes(cache);
  a.q = reinterpret_cast<const f16*>(Q);
  a.ldq = ld_q;
  a.o = O;
  a.o16 = reinterpret_cast<f16*>(O16);
  a.ldo = ld_o;
  a.lse = lse;
  a.part = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.part);
  a.stat = reinterpret_cast<float*>(static_cast<char*>(workspace) + p.stat);
  a.heads = heads;
  a.kv_heads = cache->kv_heads;
  a.ratio = heads / cache->kv_heads;
  a.rows = p.rows;
  a.rts = p.rts;
  a.window = window;
  a.groups = p.groups;
  a.whole = (int64_t)seqs->width * cache->page <= kWholeTokens;
  // (a factor of 0 would make masked scores no numbers: 2^-100 leaves every score 0 as well)
  a.flip = scale < 0.f ? 0x80008000u : 0u;
  a.c = fmaxf(fabsf(scale) * 1.44269504088896341f, 0x1p-100f);
  by_bits<Attend>(cache, a, cache->head_dim, stream);
  return hip_status(hipGetLastError());
}

}  // extern "C"
