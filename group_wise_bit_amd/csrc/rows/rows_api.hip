// Entry points of qlin_rows.h: host checks, workspace layout, launches.
#include <hip/hip_runtime.h>

#include "../../../include/qlin_rows.h"
#include "../checks.h"
#include "group.h"
#include "route.h"
#include "rows_plan.h"

using namespace qlin;

namespace {

inline bool aligned4(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 3u) == 0; }

constexpr int64_t kMaxPairs = 1 << 26;

int64_t align256(int64_t b) { return (b + 255) & ~(int64_t)255; }

// The workspace of one call, cut into 256-byte aligned parts behind the
// counters that the other entry points keep at its start.
struct Arena {
  char* base;
  int64_t at = kCounterBytes;
  template <typename T>
  T* take(int64_t count) {
    T* p = reinterpret_cast<T*>(base + at);
    at += align256(count * (int64_t)sizeof(T));
    return p;
  }
};

// Row tiles of `height` rows that `count` rows over `buckets` buckets can need.
int64_t tile_bound(int64_t count, int buckets, int height) {
  return count / height + (count < buckets ? count : buckets);
}

RowPlan take_plan(Arena& ar, int64_t count, int buckets, int height) {
  RowPlan p;
  p.order = ar.take<int32_t>(count);
  p.tiles = ar.take<int4>(tile_bound(count, buckets, height));
  p.ntiles = ar.take<int32_t>(1);
  return p;
}

// Scratch of the grouping of `count` ids: its work-groups' counts.
int32_t* take_counts(Arena& ar, int64_t count, int buckets) {
  return count > kPlanIds ? ar.take<int32_t>((int64_t)kPlanGroups * (buckets + 1)) : nullptr;
}

void run_plan(const int32_t* ids, int count, int buckets, int rows, int32_t* counts, RowPlan plan,
              hipStream_t st) {
  const int share = plan_share(count), groups = (count + share - 1) / share;
  if (counts != nullptr)
    hipLaunchKernelGGL(k_rows_count, dim3(groups), dim3(1024), 0, st, ids, count, buckets, counts);
  hipLaunchKernelGGL(k_rows_plan, dim3(groups), dim3(kPlanWaves * 64), 0, st, ids, count, buckets,
                     rows, counts, plan);
}

int64_t code_words(const qlin_weight* w) { return packed_bytes(w->n, w->k, w->bits) / 4; }

void set_weight(RowsArgs& a, int i, const qlin_weight* w) {
  a.codes[i] = static_cast<const uint32_t*>(w->data);
  a.scale[i] = w->scale;
  a.zero[i] = w->zero;
  a.code_step = code_words(w);
  a.meta_step = meta_entries(w->n, w->k, w->group);
  a.n = w->n;
  a.kb = w->k / kBlock;
  a.G = w->group == w->k ? 1 : a.kb;
}

void run_rows(const RowsArgs& a, int bits, int mode, RowsCfg c, hipStream_t st) {
  switch (bits) {
    case 2: launch_rows<2>(a, mode, c, st); break;
    case 3: launch_rows<3>(a, mode, c, st); break;
    case 4: launch_rows<4>(a, mode, c, st); break;
    case 5: launch_rows<5>(a, mode, c, st); break;
    case 6: launch_rows<6>(a, mode, c, st); break;
    case 7: launch_rows<7>(a, mode, c, st); break;
    default: launch_rows<8>(a, mode, c, st); break;
  }
}

bool stack_overlaps(const qlin_weight* w, int64_t experts, Range r) {
  const int64_t me = meta_entries(w->n, w->k, w->group) * experts;
  return overlaps(r, range_of(w->data, packed_bytes(w->n, w->k, w->bits) * experts)) ||
         overlaps(r, range_of(w->scale, me * 2)) || overlaps(r, range_of(w->zero, me));
}

// ---------------------------------------------------------------- experts --
// Up to this many (token, slot) pairs, and up to this many bytes of codes if no
// two of them share an expert, each pair reads its expert's weights by itself: no
// plan, and a token's slots are added by the work-group that multiplies them.
// Alone : grouped, 64 experts of 2048 x 1024 at 4 bits (3.4 MB each) took
// 14 : 20 us for 8 pairs, 38 : 35 us for 32, 70 : 51 us for 64; 8 of 4096 x 1792
// at 8 bits (22 MB) 25 : 27 us for 4 pairs, 43 : 42 us for 8, 75 : 48 us for 16.
constexpr int kDirectPairs = 32;
constexpr int64_t kDirectBytes = 112 << 20;

// From this many rows per expert on 64-row tiles are used, if tiled_form()
// agrees: 32-row : 64-row tiles, 64 experts of 2048 x 1024 at 4 bits 75 : 83 us at
// 8 rows each, 92 : 85 us at 16, 117 : 114 us at 32, 151 : 118 us at 48; 16 of 4096 x
// 1792 at 8 bits 93 : 95 us at 8, 104 : 96 us at 16, 142 : 111 us at 32; 128 of 1024 x
// 512 at 3 bits 50 : 53 us at 8, 61 : 62 us at 16.
constexpr int kTiledRows = 16;

struct MoePlan {
  int64_t pairs;
  bool direct;
  RowsCfg up, down;    // forms of the two products
  RowPlan rows;
  int32_t* counts;
  uint16_t* h;         // [pairs][inner] in two halves
  float* d;
  int64_t bytes;
};

MoePlan moe_plan(const qlin_weight* gate, const qlin_weight* down, int experts, int m, int64_t ld_x,
                 int top_k, void* ws) {
  const int inner = gate->n, model = gate->k;
  MoePlan p{};
  p.pairs = (int64_t)m * top_k;
  p.direct = p.pairs <= kDirectPairs &&
             p.pairs * (2 * packed_bytes(inner, model, gate->bits) +
                        packed_bytes(model, inner, down->bits)) <= kDirectBytes;
  const bool tiled = p.pairs >= kTiledRows * (int64_t)experts &&
                     tiled_form(inner, kSwiglu, p.pairs / 64 + experts / 2, m, ld_x, model);
  const int height = p.direct ? 1 : tiled ? 64 : 32;
  p.up.height = p.down.height = height;
  const int ki = inner / kBlock, km = model / kBlock;
  if (p.direct) {
    p.up.tiles = (int)p.pairs;
    p.down.tiles = m;
    gemv_form(p.up, km, p.pairs * 4 * tiles_of(inner));
    gemv_form(p.down, top_k * ki, (int64_t)m * 4 * tiles_of(model));
  } else {
    p.up.tiles = p.down.tiles = (int)tile_bound(p.pairs, experts, height);
    const int64_t used = p.pairs < experts ? p.pairs : experts;   // at most
    ksplit_form(p.up, tiles_of(inner) * used);
    ksplit_form(p.down, tiles_of(model) * used);
  }
  Arena ar{static_cast<char*>(ws)};
  p.h = ar.take<uint16_t>(2 * p.pairs * inner);
  if (!p.direct) {
    p.rows = take_plan(ar, p.pairs, experts, 32);    // (enough for 64-row tiles)
    p.counts = take_counts(ar, p.pairs, experts);
    p.d = ar.take<float>(p.pairs * model);
  }
  p.bytes = ar.at;
  return p;
}

qlin_status check_moe(const qlin_weight* gate, const qlin_weight* up, const qlin_weight* down,
                      int32_t experts, int32_t m, int32_t top_k) {
  const qlin_weight* w[3] = {gate, up, down};
  for (const qlin_weight* x : w) {
    const qlin_status st = check_weight(x, false, false);
    if (st != QLIN_OK) return st;
  }
  if (up->n != gate->n || up->k != gate->k || down->n != gate->k || down->k != gate->n)
    return QLIN_ERR_SHAPE;
  if (up->bits != gate->bits || up->group != gate->group) return QLIN_ERR_FORMAT;
  if (experts < 1 || experts > kMaxExperts || top_k < 1 || top_k > kMaxTopK || m < 0 ||
      m > kMaxM || (int64_t)m * top_k > kMaxPairs)
    return QLIN_ERR_SHAPE;
  return QLIN_OK;
}

// --------------------------------------------------------------- adapters --
// Rows are ordered by adapter if m * rank reaches this, and always for 64-row
// tiles: A x is then formed on the matrix cores, 16 rows of one adapter at a time,
// and a tile of the product holds few adapters.  Below, each row reads its own
// adapter.  Rows as they come : ordered, rank 64 on 2048 x 2048 25 : 28 us for 256
// rows, 40 : 34 us for 512; rank 16 on 4096 x 4096 58 : 66 us for 512; rank 8 on 896
// x 4864 41 : 47 us for 1024.
constexpr int64_t kSortRanks = 20480;

struct LoraPlan {
  RowsCfg cfg;
  bool sorted;         // rows are ordered by adapter first
  RowPlan rows;
  int32_t* counts;
  int tiles;           // (sorted) 16-row tiles of one adapter, at most
  int splits, steps;   // K splits of A x, 128-column steps of each
  float* t;
  int rp;
  int64_t bytes;
};

LoraPlan lora_plan(const qlin_weight* w, const qlin_adapters* ad, int m, int64_t ld_x, void* ws) {
  LoraPlan p{};
  const bool tiled = tiled_form(w->n, kLora, (m + 63) / 64, m, ld_x, w->k);
  p.cfg.height = tiled ? 64 : 32;
  p.cfg.tiles = (m + p.cfg.height - 1) / p.cfg.height;
  ksplit_form(p.cfg, tiles_of(w->n) * p.cfg.tiles);
  p.rp = (ad->rank + 15) / 16 * 16;
  p.sorted = tiled || (int64_t)m * ad->rank >= kSortRanks;
  p.cfg.dots = !p.sorted && ad->rank <= kDotRank;
  p.splits = 1;
  const int steps = (w->k + 127) / 128;
  p.steps = steps;
  Arena ar{static_cast<char*>(ws)};
  if (p.sorted) {
    p.tiles = (int)tile_bound(m, ad->slots, 16);
    // enough work-groups for the chip, a step for every wave of each
    while (p.splits < 8 && p.tiles * p.splits < 256 && steps >= 16 * p.splits) p.splits *= 2;
    p.steps = (steps + p.splits - 1) / p.splits;
    p.splits = (steps + p.steps - 1) / p.steps;
    p.rows = take_plan(ar, m, ad->slots, 16);
    p.counts = take_counts(ar, m, ad->slots);
  }
  p.t = ar.take<float>((int64_t)p.splits * m * p.rp);
  p.bytes = ar.at;
  return p;
}

qlin_status check_lora(const qlin_weight* w, const qlin_adapters* ad, int32_t m) {
  const qlin_status st = check_weight(w, false, false);
  if (st != QLIN_OK) return st;
  if (ad == nullptr) return QLIN_ERR_NULL;
  if (ad->slots < 1 || ad->slots > kMaxExperts || ad->rank < 8 || ad->rank > 128 ||
      ad->rank % 8 != 0 || m < 0 || m > kMaxM)
    return QLIN_ERR_SHAPE;
  return QLIN_OK;
}

}  // namespace

extern "C" {

qlin_status qlin_route(const qlin_router* r, const float* logits, int32_t m, int64_t ld,
                       int32_t* ids, float* weights, hipStream_t stream) {
  if (r == nullptr) return QLIN_ERR_NULL;
  if (r->experts < 1 || r->experts > kMaxExperts || r->top_k < 1 || r->top_k > kMaxTopK ||
      r->top_k > r->experts || r->groups < 1 || r->groups > 64 || r->experts % r->groups != 0 ||
      r->top_groups < 1 || r->top_groups > r->groups || r->group_top < 1 || r->group_top > 2 ||
      r->top_groups * (r->experts / r->groups) < r->top_k)
    return QLIN_ERR_SHAPE;
  if ((r->score != QLIN_SCORE_SOFTMAX && r->score != QLIN_SCORE_SIGMOID) ||
      (r->renormalize != 0 && r->renormalize != 1))
    return QLIN_ERR_FORMAT;
  if (m < 0 || m > kMaxM || ld < r->experts) return QLIN_ERR_SHAPE;
  if (m == 0) return QLIN_OK;
  if (logits == nullptr || ids == nullptr || weights == nullptr) return QLIN_ERR_NULL;
  if (!aligned4(logits) || !aligned4(ids) || !aligned4(weights) || !aligned4(r->bias))
    return QLIN_ERR_ALIGN;
  const Range in[2] = {range_of(logits, ((int64_t)(m - 1) * ld + r->experts) * 4),
                       range_of(r->bias, r->bias != nullptr ? (int64_t)r->experts * 4 : 0)};
  const Range out[2] = {range_of(ids, (int64_t)m * r->top_k * 4),
                        range_of(weights, (int64_t)m * r->top_k * 4)};
  for (const Range& o : out)
    for (const Range& i : in)
      if (overlaps(o, i)) return QLIN_ERR_ALIAS;
  if (overlaps(out[0], out[1])) return QLIN_ERR_ALIAS;
  const qlin_status st = check_device();
  if (st != QLIN_OK) return st;
  RouteArgs a{logits, r->bias, ld, ids, weights, m, r->experts, r->top_k, r->groups,
              r->top_groups, r->group_top, r->scale, r->score == QLIN_SCORE_SIGMOID,
              r->renormalize != 0};
  const dim3 grid((m + kRouteWaves - 1) / kRouteWaves), block(kRouteWaves * 64);
  if (r->experts <= 64) hipLaunchKernelGGL((k_route<1>), grid, block, 0, stream, a);
  else if (r->experts <= 128) hipLaunchKernelGGL((k_route<2>), grid, block, 0, stream, a);
  else if (r->experts <= 256) hipLaunchKernelGGL((k_route<4>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((k_route<8>), grid, block, 0, stream, a);
  return hip_status(hipGetLastError());
}

int64_t qlin_moe_mlp_workspace_bytes(const qlin_weight* gate, const qlin_weight* down,
                                     int32_t experts, int32_t m, int32_t top_k) {
  if (check_moe(gate, gate, down, experts, m, top_k) != QLIN_OK || m == 0) return 0;
  return moe_plan(gate, down, experts, m, gate->k, top_k, nullptr).bytes;
}

qlin_status qlin_moe_mlp(const qlin_weight* gate, const qlin_weight* up, const qlin_weight* down,
                         int32_t experts, const uint16_t* X, int32_t m, int64_t ld_x,
                         const int32_t* ids, const float* weights, int32_t top_k, float* Y,
                         uint16_t* Y16, int64_t ld_y, void* workspace, int64_t workspace_bytes,
                         hipStream_t stream) {
  qlin_status st = check_moe(gate, up, down, experts, m, top_k);
  if (st != QLIN_OK) return st;
  if (ld_x < gate->k || ld_y < down->n) return QLIN_ERR_SHAPE;
  if (ld_x % 8 != 0) return QLIN_ERR_ALIGN;
  if (m == 0) return QLIN_OK;
  if (X == nullptr || ids == nullptr || weights == nullptr || (Y == nullptr && Y16 == nullptr))
    return QLIN_ERR_NULL;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(Y16) || !aligned4(ids) || !aligned4(weights) ||
      !aligned16(workspace))
    return QLIN_ERR_ALIGN;
  const int inner = gate->n, model = gate->k;
  const MoePlan p = moe_plan(gate, down, experts, m, ld_x, top_k, workspace);
  if (!rows_fits(inner, kSwiglu, p.up) || !rows_fits(model, kDown, p.down)) return QLIN_ERR_SHAPE;
  if (workspace == nullptr || workspace_bytes < p.bytes) return QLIN_ERR_WORKSPACE;
  const int64_t span = (int64_t)(m - 1) * ld_y + model;
  const Range out[3] = {range_of(workspace, workspace_bytes),
                        range_of(Y, Y != nullptr ? span * 4 : 0),
                        range_of(Y16, Y16 != nullptr ? span * 2 : 0)};
  const Range in[3] = {range_of(X, ((int64_t)(m - 1) * ld_x + model) * 2),
                       range_of(ids, p.pairs * 4), range_of(weights, p.pairs * 4)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i], r)) return QLIN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return QLIN_ERR_ALIAS;
    if (stack_overlaps(gate, experts, out[i]) || stack_overlaps(up, experts, out[i]) ||
        stack_overlaps(down, experts, out[i]))
      return QLIN_ERR_ALIAS;
  }
  st = check_device();
  if (st != QLIN_OK) return st;
  if (!p.direct)
    run_plan(ids, (int)p.pairs, experts, p.up.height, p.counts, p.rows, stream);
  RowsArgs a{};
  set_weight(a, 0, gate);
  set_weight(a, 1, up);
  a.X = X;
  a.ldx = ld_x;
  a.m = m;
  a.top_k = top_k;
  a.plan = p.rows;
  a.experts = experts;
  a.ids = ids;
  a.y16 = p.h;
  a.ldy = 2 * (int64_t)inner;
  run_rows(a, gate->bits, kSwiglu, p.up, stream);
  RowsArgs b{};
  set_weight(b, 0, down);
  b.X = p.h;
  b.ldx = 2 * (int64_t)inner;
  b.m = m;
  b.top_k = top_k;
  b.plan = p.rows;
  b.experts = experts;
  b.ids = ids;
  b.weights = weights;
  if (p.direct) {
    b.y = Y;
    b.y16 = Y16;
    b.ldy = ld_y;
    run_rows(b, down->bits, kToken, p.down, stream);
    return hip_status(hipGetLastError());
  }
  b.y = p.d;
  b.ldy = model;
  run_rows(b, down->bits, kDown, p.down, stream);
  const int64_t groups = ((int64_t)m * (model / 4) + 255) / 256;
  hipLaunchKernelGGL(k_rows_combine, dim3((unsigned)(groups < 65536 ? groups : 65536)), dim3(256),
                     0, stream, p.d, ids, m, top_k, experts, model, Y, Y16, ld_y);
  return hip_status(hipGetLastError());
}

int64_t qlin_gemm_lora_workspace_bytes(const qlin_weight* w, const qlin_adapters* ad, int32_t m) {
  if (check_lora(w, ad, m) != QLIN_OK || m == 0) return 0;
  // (a larger stride of X never needs more)
  return lora_plan(w, ad, m, w->k, nullptr).bytes;
}

qlin_status qlin_gemm_lora(const qlin_weight* w, const qlin_adapters* ad, const uint16_t* X,
                           int32_t m, int64_t ld_x, const int32_t* ids, float* Y, uint16_t* Y16,
                           int64_t ld_y, void* workspace, int64_t workspace_bytes,
                           hipStream_t stream) {
  qlin_status st = check_lora(w, ad, m);
  if (st != QLIN_OK) return st;
  if (ld_x < w->k || ld_y < w->n) return QLIN_ERR_SHAPE;
  if (ld_x % 8 != 0) return QLIN_ERR_ALIGN;
  if (m == 0) return QLIN_OK;
  if (X == nullptr || ids == nullptr || ad->a == nullptr || ad->b == nullptr ||
      (Y == nullptr && Y16 == nullptr))
    return QLIN_ERR_NULL;
  if (!aligned16(X) || !aligned16(Y) || !aligned16(Y16) || !aligned16(ad->a) ||
      !aligned16(ad->b) || !aligned4(ad->scale) || !aligned4(ids) || !aligned16(workspace))
    return QLIN_ERR_ALIGN;
  const LoraPlan p = lora_plan(w, ad, m, ld_x, workspace);
  if (!rows_fits(w->n, kLora, p.cfg)) return QLIN_ERR_SHAPE;
  if (workspace == nullptr || workspace_bytes < p.bytes) return QLIN_ERR_WORKSPACE;
  const int64_t span = (int64_t)(m - 1) * ld_y + w->n;
  const int64_t sr = (int64_t)ad->slots * ad->rank;
  const Range out[3] = {range_of(workspace, workspace_bytes),
                        range_of(Y, Y != nullptr ? span * 4 : 0),
                        range_of(Y16, Y16 != nullptr ? span * 2 : 0)};
  const Range in[5] = {range_of(X, ((int64_t)(m - 1) * ld_x + w->k) * 2),
                       range_of(ids, (int64_t)m * 4), range_of(ad->a, sr * w->k * 2),
                       range_of(ad->b, sr * w->n * 2),
                       range_of(ad->scale, ad->scale != nullptr ? (int64_t)ad->slots * 4 : 0)};
  for (int i = 0; i < 3; ++i) {
    for (const Range& r : in)
      if (overlaps(out[i], r)) return QLIN_ERR_ALIAS;
    for (int j = 0; j < i; ++j)
      if (overlaps(out[i], out[j])) return QLIN_ERR_ALIAS;
    if (output_overlaps_weight(w, out[i])) return QLIN_ERR_ALIAS;
  }
  st = check_device();
  if (st != QLIN_OK) return st;
  ShrinkArgs s{};
  s.X = X;
  s.ldx = ld_x;
  s.m = m;
  s.k = w->k;
  s.slots = ad->slots;
  s.rank = ad->rank;
  s.rp = p.rp;
  s.ids = ids;
  s.a = ad->a;
  s.scale = ad->scale;
  s.t = p.t;
  if (p.sorted) {
    s.plan = p.rows;
    s.splits = p.splits;
    s.steps = p.steps;
    run_plan(ids, m, ad->slots, 16, p.counts, p.rows, stream);
    const dim3 grid(p.tiles * p.splits), block(512);
    if (p.rp <= 16) hipLaunchKernelGGL((k_lora_shrink_tile<1>), grid, block, 0, stream, s);
    else if (p.rp <= 32) hipLaunchKernelGGL((k_lora_shrink_tile<2>), grid, block, 0, stream, s);
    else if (p.rp <= 64) hipLaunchKernelGGL((k_lora_shrink_tile<4>), grid, block, 0, stream, s);
    else hipLaunchKernelGGL((k_lora_shrink_tile<8>), grid, block, 0, stream, s);
  } else {
    hipLaunchKernelGGL(k_lora_shrink_row, dim3(m, p.rp / 8), dim3(512), 0, stream, s);
  }
  RowsArgs a{};
  set_weight(a, 0, w);
  a.X = X;
  a.ldx = ld_x;
  a.m = m;
  a.top_k = 1;
  a.y = Y;
  a.y16 = Y16;
  a.ldy = ld_y;
  a.ids = ids;
  a.t = p.t;
  a.tsplits = p.splits;
  if (p.sorted) a.plan = p.rows;
  a.b = ad->b;
  a.slots = ad->slots;
  a.rank = ad->rank;
  a.rp = p.rp;
  run_rows(a, w->bits, kLora, p.cfg, stream);
  return hip_status(hipGetLastError());
}

}  // extern "C"
