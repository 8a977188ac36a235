/*
 * qlin cache of keys and values, held in group-wise affine codes in pages:
 * quantizing new tokens into it, reading tokens back, and attention of one new
 * token per sequence over it.  Part of libqlin; status codes, memory ownership,
 * alignment (16 bytes, except where noted) and stream capture rules are those of
 * qlin.h.  Every call enqueues kernels on the caller's stream and returns without
 * synchronizing; lengths, page numbers and row offsets are read on the GPU only.
 * All of a call's pointers must belong to the current device.
 *
 * What a token is in the cache.  The head_dim values of a key (or value) of one
 * head are cut into groups of 64.  With 4 or 8 bits a group has
 *     lo = min(w, 0),  hi = max(w, 0) over its values,  qmax = 2^bits - 1,
 *     s = fp16( fl32( fl32(hi - lo) / qmax ) ),
 *     z = clamp( rint( fl32(-lo / s) ), 0, qmax ),
 *     q = clamp( rint( fl32(w / s) ) + z, 0, qmax ),
 * rint rounding half-way cases to even, and stands for s * (q - z).  That is
 * qlin_quantize's rounding over a range that holds 0, so that a group of one sign
 * is as close as any other (s / 2, and what z's and s's rounding add).  A group whose stored scale is 0
 * reads as zeros; one that holds an infinity or NaN gets the scale NaN and reads as NaN.
 * With 16 bits the values are kept as they are.
 *
 * ---------------------------------------------------------------------------
 * Layout of a page.  A page holds `page` tokens of every head of keys and
 * values; [pages][kv_heads][page / 32] tiles of 32 tokens follow one another, each
 *     key codes, value codes, key scales, value scales, key zeros, value zeros
 * (scales and zeros only with fewer than 16 bits).  With G = head_dim / 64, for
 * token t of the tile (half h = t / 16) and dim x (group c = x / 64, y = x % 64):
 *   key codes, 4 * head_dim * bits bytes: 64 lanes, lane = 16 * (y / 16) + t % 16;
 *     a lane's run holds its codes in the order i = (h * G + c) * 16 + y % 16, 32 /
 *     bits to a word, code i at bit 16 * (i % 2) + bits * (i % (32 / bits) / 2)
 *     of word i / (32 / bits); word w of the run lies at word (w / 4 * 64 + lane) * 4 + w % 4.
 *   value codes, 4 * head_dim * bits bytes: lane = 16 * (t % 16 / 4) + y / 4; with
 *     n = 16 / bits codes to a half-word, the code is at bit
 *     16 * (t % 2) + bits * (y % 4 % n) of word
 *     ((c * (4 / n) + y % 4 / n) * 64 + lane) * 4 + 2 * h + t % 4 / 2.
 *   scales, fp16 [G][4][2][4] for keys and for values: [c][t % 16 / 4][h][t % 4].
 *   zeros, uint8: keys [16][2][G]: [t % 16][h][c]; values [4][G][2][4]:
 *     [t % 16 / 4][c][h][t % 4].
 * So a wave reads a tile in whole 16-byte units of its lanes, in the order in which the
 * matrix cores take keys and values, and a token is written without reading its neighbours.
 * ---------------------------------------------------------------------------
 */
#ifndef QLIN_KV_H
#define QLIN_KV_H

#include "qlin.h"

#ifdef __cplusplus
extern "C" {
#endif

/* A cache of one layer. */
typedef struct qlin_kv_cache {
  int32_t pages;            /* 1 .. 2^31 - 1                                     */
  int32_t kv_heads;         /* 1 .. 256                                          */
  int32_t head_dim;         /* 64, 128 or 256                                    */
  int32_t page;             /* tokens per page: 32, 64, 128 or 256               */
  int32_t k_bits, v_bits;   /* 4, 8 or 16 each                                   */
  void* data;               /* pages * kv_heads * qlin_kv_page_bytes bytes       */
} qlin_kv_cache;

/* The sequences of a batch.  Sequence b has lengths[b] tokens; token p lies in
 * page table[b * ld + p / cache.page].  A length below 1 is an empty sequence. A
 * token beyond the table, or in a page that is not 0 .. pages - 1, is not there.
 * Work-groups find their sequence by the lengths of all (rows with starts; attention with
 * tables above 1024 tokens), so that such a call's time grows with the square of seqs from some
 * thousands on: with one token and one head of 64 each, 1024 sequences take 13 us to write and
 * 25 to attend to, 4096 102 and 104, 16384 1360 and 860. */
typedef struct qlin_kv_seqs {
  int32_t seqs;             /* 0 .. 65536                                        */
  int32_t width;            /* pages per table row, width * cache.page <= 2^27   */
  const int32_t* table;     /* device [seqs, ld], 4-byte aligned                 */
  int64_t ld;               /* >= width                                          */
  const int32_t* lengths;   /* device [seqs], 4-byte aligned                     */
} qlin_kv_seqs;

/* Bytes of one page of one head (0 if invalid). */
int64_t qlin_kv_page_bytes(int32_t head_dim, int32_t page, int32_t k_bits, int32_t v_bits);

/*
 * New tokens enter the cache.  Rows starts[b] .. starts[b + 1] - 1 of K and V are
 * the last tokens of sequence b (its length counts them already); starts: device
 * int32 [seqs + 1], ascending from 0 on, 4-byte aligned; NULL: row b is the last token of
 * sequence b, and m >= seqs.  Rows from starts[seqs] on (padding) are not read.
 *   K, V   fp16 [m, ld_k] and [m, ld_v], a row kv_heads * head_dim values, pitches
 *          multiples of 8.
 * A token whose position is negative, or that is not there, is left out.  Nothing
 * but the written tokens changes in a page.  Two rows of a call must not go to the same place (a page
 * that is written belongs to one sequence): what such a place then holds is undefined.
 * m <= 2^20; seqs = 0 or m = 0 is a no-op.  A call whose grid would have 2^32 threads is
 * refused with QLIN_ERR_SHAPE: (m / 32 + 2 min(m, seqs)) * ceil(kv_heads * (2 + head_dim / 64) / 4),
 * without starts seqs times the second factor, is below 2^24.
 */
qlin_status qlin_kv_write(const qlin_kv_cache* cache, const uint16_t* K, int64_t ld_k,
                          const uint16_t* V, int64_t ld_v, int32_t m, const qlin_kv_seqs* seqs,
                          const int32_t* starts, hipStream_t stream);

/*
 * Tokens read back: rows starts[b] .. starts[b + 1] - 1 of K and V become the last
 * tokens of sequence b (starts as for qlin_kv_write; NULL: row b the last token of b),
 * each value s * (q - z).  K and V are both fp16 (wide = 0: rounded to nearest even, +-65504 at
 * most unless the value is kept with 16 bits) or both fp32 (wide = 1: exact), [m, ld_k] and [m, ld_v],
 * pitches multiples of 8 (K and V may be columns of one matrix).  Rows of tokens that
 * are not there are zero; rows from starts[seqs] on are not written.  Limits as for qlin_kv_write.
 */
qlin_status qlin_kv_read(const qlin_kv_cache* cache, const qlin_kv_seqs* seqs,
                         const int32_t* starts, int32_t m, void* K, int64_t ld_k, void* V,
                         int64_t ld_v, int32_t wide, hipStream_t stream);

/*
 * Attention of one new token per sequence over its cached tokens:
 *     S[p] = scale * q . k_p,   P = softmax(S),   O = sum_p P[p] v_p,
 *     lse = log( sum_p exp(S[p]) ),
 * p over the tokens of the sequence that are there, with window > 0 over those from lengths[b] -
 * window on.  heads is a multiple of kv_heads; head i of Q reads head
 * i / (heads / kv_heads) of the cache.
 *   Q    fp16 [seqs, ld_q], a row heads * head_dim values, ld_q % 8 == 0.
 *   O    fp32, O16 the same rounded to fp16 (nearest even): [seqs, ld_o], ld_o >=
 *        heads * head_dim, % 8 == 0; either may be NULL, not both.
 *   lse  fp32 [seqs, heads] contiguous, 4-byte aligned, or NULL.
 * A row without tokens (or whose scores are all -inf) is zero, its lse -inf.
 * What lies in masked places (behind a sequence's end, before its window, in
 * pages that are not in the table) does not matter, NaN included.  Of the tokens that are
 * seen, one whose score is -inf weighs nothing; a score of +inf or NaN makes its row not finite,
 * and so does a value that is not finite, in its dims, whatever its token weighs.
 * Keys and values enter as the exact values of their codes; sums, the
 * softmax's statistics and scales are held in fp32, P * s (s the scale of the value's
 * group, 1 with 16 bits; what is below counts as 2^-24) to 2^-22 of it, rounded to
 * nearest, or to 2^-39 of the row's largest where that is more.
 * Deterministic: the result depends on the inputs and, to the order of fp32 sums,
 * on the lengths of all the call's sequences.
 * The cache is read once for every 16 query heads of a head of the cache: the tokens of all
 * sequences are dealt out evenly over the work-groups, and the parts of a sequence joined in a
 * second kernel (tables of up to 1024 tokens: neither).
 * workspace: scratch of qlin_kv_attention_workspace_bytes (or QLIN_ERR_WORKSPACE; 0
 * is returned there for invalid arguments); its first 65536 bytes are left as they
 * are, so that it may be the buffer of the other calls.  Calls that can run at the same time need
 * workspaces of their own.  heads <= 1024; |scale| <= 2^20; seqs * heads < 2^24.
 */
int64_t qlin_kv_attention_workspace_bytes(const qlin_kv_cache* cache, const qlin_kv_seqs* seqs,
                                          int32_t heads);
qlin_status qlin_kv_attention(const qlin_kv_cache* cache, const qlin_kv_seqs* seqs,
                              const uint16_t* Q, int64_t ld_q, int32_t heads, float scale,
                              int32_t window, float* O, uint16_t* O16, int64_t ld_o, float* lse,
                              void* workspace, int64_t workspace_bytes, hipStream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* QLIN_KV_H */
