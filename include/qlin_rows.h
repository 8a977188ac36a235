/*
 * qlin products whose weights differ from row to row of a batch: routing to
 * experts, the experts' gated MLP over packed weights, and low-rank adapters
 * of many requests beside one packed projection.  Part of libqlin; the types,
 * status codes, packed layout, memory ownership, alignment (16 bytes, except
 * where noted) and stream capture rules are those of qlin.h.  Every call
 * enqueues kernels on the caller's stream and returns without synchronizing;
 * nothing about the ids is read on the host.  All of a call's pointers must
 * belong to the current device.  m = 0 is a no-op in every call (pointers are
 * then not looked at).  A product whose grid would have 2^32 threads is refused
 * with QLIN_ERR_SHAPE (rows, one per token and slot, times columns: none below 2^32).
 *
 * Workspaces.  A call's workspace is scratch: nothing in it is kept between
 * calls, and it needs no initialization, with one exception that lets it be
 * the buffer that qlin_gemm and the others share: its first 65536 bytes are
 * left as they are.  Calls that can run at the same time (other streams, two
 * captured graphs) need workspaces of their own, and so do calls that two
 * threads enqueue on one stream at the same time: a call's kernels hand their
 * results on in its workspace.
 */
#ifndef QLIN_ROWS_H
#define QLIN_ROWS_H

#include "qlin.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  QLIN_SCORE_SOFTMAX = 0,   /* p = exp(l - max) / sum over the row's experts     */
  QLIN_SCORE_SIGMOID = 1    /* p = 1 / (1 + exp(-l)), every expert on its own    */
};

/* How a router turns logits into experts and weights. */
typedef struct qlin_router {
  int32_t experts;          /* 1 .. 512                                          */
  int32_t top_k;            /* experts per row, 1 .. 32                          */
  int32_t score;            /* QLIN_SCORE_*                                      */
  int32_t groups;           /* experts are cut into this many equal groups,
                               1 .. 64, experts % groups == 0                    */
  int32_t top_groups;       /* groups kept per row, 1 .. groups; they must hold
                               top_k experts                                     */
  int32_t group_top;        /* a group's value: the sum of its 1 or 2 best
                               biased scores                                     */
  int32_t renormalize;      /* 0 / 1: divide the chosen scores by their sum      */
  float scale;              /* multiplies the weights                            */
  const float* bias;        /* fp32 [experts] or NULL: added to the scores for
                               the choice, not to the weights                    */
} qlin_router;

/*
 * Routing to experts, one row of logits per token:
 *     p = softmax or sigmoid of the row,   b = p + bias,
 *     kept groups: the top_groups groups of largest value (only if groups > 1),
 *     ids[i, :] = the top_k experts of largest b in the kept groups, descending,
 *     weights[i, j] = scale * p[ids] (/ sum_j p[ids] if renormalize).
 * logits fp32 [m, ld], ld >= experts (any alignment to 4 bytes); ids int32 and
 * weights fp32 [m, top_k], contiguous, 4-byte aligned.
 * The choice is that of 64-bit arithmetic on the fp32 logits and bias; without
 * a bias experts are ordered by their logits, which is the order of the exact
 * scores.  Equal values go to the lowest index, among groups too.  Weights
 * are correct to a few units of fp32, however far below the row's largest logit
 * the chosen ones lie (scores are 64-bit values: they are whole down to 2^-1022,
 * exp(-708), and 0 from about exp(-745) on).
 * Masked experts: a logit of -inf or NaN, or a bias of -inf or NaN, takes the
 * expert out of the row (and, a logit, out of the softmax's sum); +inf counts
 * as the largest finite logit.  A row with fewer than top_k experts left has
 * id -1 and weight 0 in its remaining places.  If the chosen scores sum to 0,
 * renormalized weights are 0.
 */
qlin_status qlin_route(const qlin_router* r, const float* logits, int32_t m, int64_t ld,
                       int32_t* ids, float* weights, hipStream_t stream);

/*
 * The experts' gated MLP over packed weights:
 *     Y[i, :] = sum_j weights[i, j] * down_e( silu(gate_e x_i) * up_e x_i ),
 *     e = ids[i, j],  j = 0 .. top_k - 1,
 * A stack of experts is described by the qlin_weight of expert 0 and the
 * number of experts: expert e's codes, scales and zeros lie e times
 * qlin_packed_bytes / qlin_meta_entries after expert 0's (the buffers of one
 * qlin_quantize after the other).  gate and up: PACKED, the same n (the inner
 * size), k (the model size), bits and group; down: n = gate.k, k = gate.n, its
 * own bits and group (64, or its k).  The inner size is a multiple of 64.
 * X fp16 [m, ld_x] (ld_x >= gate.k, % 8 == 0); ids int32 and weights fp32
 * [m, top_k] contiguous, 4-byte aligned, as qlin_route writes them: an id
 * outside [0, experts) contributes nothing (its weight is not read), and a row
 * without experts is zero.  An expert may stand in a row twice.
 * experts <= 512, top_k <= 32, m * top_k <= 2^26.
 * Outputs, either may be NULL (not both), leading dimension ld_y >= down.n for
 * both: Y fp32, Y16 the same rounded to fp16 (nearest even).
 * Every product x * (q - z) is exact, scales are applied and sums held in fp32;
 * silu(g) * u enters the down projection with 22 bits (in steps of 2^-24 below
 * 2^-3; it is infinite from 65520 on, and its row then not finite).  Deterministic: each row's result depends on its own
 * inputs and on the call's sizes and strides only.
 * workspace_bytes >= qlin_moe_mlp_workspace_bytes(gate, down, experts, m,
 * top_k), or QLIN_ERR_WORKSPACE (0 is returned there for invalid arguments).
 */
int64_t qlin_moe_mlp_workspace_bytes(const qlin_weight* gate, const qlin_weight* down,
                                     int32_t experts, int32_t m, int32_t top_k);
qlin_status qlin_moe_mlp(const qlin_weight* gate, const qlin_weight* up, const qlin_weight* down,
                         int32_t experts, const uint16_t* X, int32_t m, int64_t ld_x,
                         const int32_t* ids, const float* weights, int32_t top_k, float* Y,
                         uint16_t* Y16, int64_t ld_y, void* workspace, int64_t workspace_bytes,
                         hipStream_t stream);

/* A pool of low-rank adapters of one projection (slots of equal rank; an
 * adapter of smaller rank is padded with zeros). */
typedef struct qlin_adapters {
  int32_t slots;            /* 1 .. 512                                          */
  int32_t rank;             /* 8 .. 128, a multiple of 8                         */
  const uint16_t* a;        /* fp16 [slots, rank, k], contiguous                 */
  const uint16_t* b;        /* fp16 [slots, n, rank], contiguous                 */
  const float* scale;       /* fp32 [slots] or NULL (all 1), 4-byte aligned      */
} qlin_adapters;

/*
 * A packed projection with a low-rank adapter per row:
 *     Y[i, :] = W x_i + scale[a] * B_a (A_a x_i),   a = ids[i],
 * the base product alone where ids[i] is outside [0, slots).  w PACKED [n, k];
 * X fp16 [m, ld_x] (ld_x >= k, % 8 == 0); ids int32 [m], 4-byte aligned.
 * Outputs as for qlin_moe_mlp: Y fp32 and / or Y16 fp16, both [m, ld_y],
 * ld_y >= n.  Every product x * (q - z) and x * a is exact, scales are applied
 * and sums held in fp32; A_a x_i enters the second product with 22 bits or more.
 * Deterministic: each row's result depends on its own inputs, on the call's
 * sizes and strides and, to the order of fp32 sums, on the ids of the rows that
 * share its tile.  A row that is not finite through its adapter changes no other
 * row.
 * workspace_bytes >= qlin_gemm_lora_workspace_bytes(w, ad, m), or
 * QLIN_ERR_WORKSPACE (0 is returned there for invalid arguments).
 */
int64_t qlin_gemm_lora_workspace_bytes(const qlin_weight* w, const qlin_adapters* ad, int32_t m);
qlin_status qlin_gemm_lora(const qlin_weight* w, const qlin_adapters* ad, const uint16_t* X,
                           int32_t m, int64_t ld_x, const int32_t* ids, float* Y, uint16_t* Y16,
                           int64_t ld_y, void* workspace, int64_t workspace_bytes,
                           hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_ROWS_H */
