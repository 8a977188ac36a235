/*
 * qlin: drawing the next token of every sequence from its logits (the products of
 * the LM head, fp32) with temperature, top-k, top-p and min-p, from given random
 * numbers.  Part of libqlin; status codes, memory ownership, alignment and stream
 * capture rules are those of qlin.h, except that 4-byte alignment is enough here.
 * The call enqueues kernels on the caller's stream and returns without synchronizing;
 * settings and random numbers are read on the GPU only, one per row.
 */
#ifndef QLIN_SAMPLE_H
#define QLIN_SAMPLE_H

#include "qlin.h"

#ifdef __cplusplus
extern "C" {
#endif

/* The settings of the rows: device arrays [m], each NULL where it is off for all. */
typedef struct qlin_sampling {
  const float* temperature; /* NULL: 1.  Not above 0: the first of the largest    */
  const int32_t* top_k;     /* below 1: off                                       */
  const float* top_p;       /* not below 1: off;  0 or less: one token            */
  const float* min_p;       /* not above 0: off;  above 1: one token              */
} qlin_sampling;

/*
 * Row i of logits, fp32 [m, ld], ld >= vocab, and u[i] in [0, 1):
 *     p[j] = exp( (l[j] - max l) / temperature ),
 *     order: by logit, descending, equal logits by index, ascending;
 *     kept: the longest beginning of the order with at most top_k tokens, none behind
 *       the first that brings the sum of p to top_p times that of the first top_k, and
 *       p[j] >= min_p (the first token is always kept);
 *     ids[i] = the lowest j for which the sum of p over the kept tokens 0 .. j
 *       exceeds u[i] times that over all kept ones;
 *     probs[i] = p[ids[i]] over that sum.
 * Tokens whose logit is -inf or NaN are not there; +inf counts as the largest
 * finite logit.  A row without tokens has id -1 and probability 0.  u below 0
 * (or NaN) counts as 0, and from 1 on takes the last kept token.
 * p is formed in 64 bits; tokens below exp(-31.5) of the largest may count as 0.  The
 * choice is that of exact arithmetic but where a border (of top_p, min_p or u) lies
 * within 2^-34 + vocab * 2^-45 of it, relative to the sum.  Deterministic: a row's result
 * depends on its own logits, settings and u only.
 * ids int32 [m]; probs fp32 [m] or NULL.  1 <= vocab <= 2^18, m <= 2^20; m = 0 is a no-op.
 * workspace: scratch of qlin_sample_workspace_bytes (or QLIN_ERR_WORKSPACE; 0 is
 * returned there for invalid arguments), 16-byte aligned; its first 65536 bytes are left
 * as they are.  Calls that can run at the same time need workspaces of their own.
 */
int64_t qlin_sample_workspace_bytes(int32_t m, int32_t vocab);
qlin_status qlin_sample(const qlin_sampling* s, const float* logits, int32_t m, int32_t vocab,
                        int64_t ld, const float* u, int32_t* ids, float* probs, void* workspace,
                        int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_SAMPLE_H */
