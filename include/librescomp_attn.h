/*
 * librescomp: attention over packed sequences with keys and values in full
 * precision, and the join of attentions over different tokens.
 *
 * Next to the 8-bit cache of librescomp_kv.h: whole prompts attend to their own
 * keys and values before these are stored, a GPU of a sequence-parallel step
 * attends to its own share as it is, and the result is joined with that of
 * rc_kv_attend over the rest:
 *
 *   rc_attn_packed   attention of sequences of different lengths that lie one after
 *                    the other, without padding
 *   rc_attn_join     several attentions of the same queries over different tokens
 *                    become attention over all of them
 *
 * The conventions of librescomp_kv.h hold: device pointers owned by the caller,
 * rows as rc_kv_view_t; calls are asynchronous on the given stream, never
 * synchronise the host and may be captured; calls on one plan are serialised on
 * one stream; a rejected request launches nothing and writes nothing.
 */
#ifndef LIBRESCOMP_ATTN_H
#define LIBRESCOMP_ATTN_H

#include "librescomp_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RC_ATTN_MAX_PARTS 8    /* attentions that one rc_attn_join takes              */

typedef struct rc_attn_plan* rc_attn_plan_t; /* opaque; owns its workspace only */

typedef struct {
  int32_t q_heads;     /* query heads, a multiple of kv_heads: query head h reads    */
  int32_t kv_heads;    /*   key head h / (q_heads / kv_heads)                        */
  int32_t head_dim;    /* 64 or 128                                                  */
  int32_t max_seqs;    /* sequences of a call at most                                */
  int32_t max_queries; /* query tokens of a call at most, all sequences together     */
  int32_t max_keys;    /* key tokens of a call at most, all sequences together       */
} rc_attn_shape_t;

/* rc_attn_params_t.flags: query i of n of a sequence with m keys sees keys 0 .. m - n + i
 * (the queries are the sequence's last n tokens; the first n - m of more queries than
 * keys see none). Without it every query sees all keys of its sequence. */
#define RC_ATTN_CAUSAL 1u

typedef struct {
  float scale;         /* factor of the scores; 0: 1 / sqrt(head_dim)                */
  uint32_t flags;      /* 0 or RC_ATTN_CAUSAL                                        */
} rc_attn_params_t;

/* Validate the request and allocate the workspace (rc_attn_workspace_bytes) on the
 * current device: partial results of at most half a gigabyte, and in fp32, for calls of
 * many rows, max_keys keys and values as halves (if that is at most 4 GB; plans for more
 * keys run a slower kernel). dtype: of all tensors of the plan's calls. Errors:
 * RC_ERR_INVALID_ARG (null pointer, bad value), RC_ERR_UNSUPPORTED (a valid value that this
 * library does not implement: another head_dim, more than 65535 sequences, 32767 key heads
 * or 2^30 keys, 2^30 query rows, max_queries * q_heads, or more), RC_ERR_HIP. */
rc_status_t rc_attn_plan_create(rc_attn_shape_t shape, rc_dtype_t dtype, const rc_attn_params_t* params,
                                rc_attn_plan_t* out);

/* Attention: out = softmax(scale * q k^T) v, each query over the keys of its own
 * sequence. q, out: [q_tokens][q_heads][head_dim], k, v: [kv_tokens][kv_heads][head_dim]
 * (views of a batch of 1). Sequence b has the query tokens q_offsets[b] ..
 * q_offsets[b + 1] - 1 and the keys kv_offsets[b] .. kv_offsets[b + 1] - 1; offsets are
 * device int32 [seqs + 1] that do not descend. kv_offsets NULL: the same as q_offsets.
 * Offsets are cut to 0 .. tokens, and a sequence that ends before it starts is empty.
 * max_q, max_kv: bounds of one sequence's queries and keys that the host knows (0: all
 * tokens of the call; among thousands of sequences a block of threads then goes through all
 * offsets to find its rows); of a longer sequence only the first max_q queries and the first
 * max_kv keys are there. Rows of out and lse that belong to no sequence's queries stay
 * as they are.
 * RC_ERR_UNSUPPORTED: a call that would take 2^24 blocks of threads or more: one at least for
 * each key head of each sequence, and each 16 to 256 query rows (bound it by max_q).
 * lse (NULL, or fp32 [q_tokens][q_heads]): the natural logarithm of the sum of the
 * exponentials. A query that sees no key, or whose scores are all -infinity, gets 0 and
 * -infinity.
 * Precision: scores, sums, the running maximum and outputs are held in fp32 and rounded
 * once. In bf16 the weights may be rounded to bf16 (8 bits) for their product with v, not
 * for their sum: before the last rounding an output is within 2^-8 of the weighted mean of
 * |v|; sums of weights times values reach 2^10 times the number of keys times |v| (in fp32 the
 * number of keys times |v|), so that values of 2^100 and more may overflow. In fp32 the factors
 * of a product (q, k, v and the weights) may be taken as sums of two f16, 22 bits each, on a
 * scale of their row of head_dim values: of a row's values under 2^-17 of its largest those bits
 * are lost that lie under 2^-39 of it, of all values those under 2^-146, of weights (times the
 * largest |v| of their token) those under 2^-33 of a query's largest.
 * NaN and infinities: what a query does not see does not reach it, whatever it holds. A
 * NaN among the queries, or the keys that one sees, or a score of +infinity makes its
 * outputs and lse NaN; a value that is not finite makes the outputs that see it not finite. */
rc_status_t rc_attn_packed(rc_attn_plan_t plan, hipStream_t stream, int seqs, const int32_t* q_offsets,
                           const int32_t* kv_offsets, int q_tokens, int kv_tokens, int max_q, int max_kv,
                           const rc_kv_view_t* q, const rc_kv_view_t* k, const rc_kv_view_t* v,
                           const rc_kv_view_t* out, float* lse);

/* Free the plan and its workspace; no launched work may still use it. NULL is
 * accepted. */
rc_status_t rc_attn_plan_destroy(rc_attn_plan_t plan);

/* Device workspace that the plan owns. 0 for a NULL plan. */
size_t rc_attn_workspace_bytes(rc_attn_plan_t plan);

/* Join `parts` (1 .. RC_ATTN_MAX_PARTS) attentions of the same queries over different
 * tokens: with L = log(sum_i exp(lses[i])), out = sum_i exp(lses[i] - L) * outs[i], lse = L.
 * outs: host array of views of [batch][tokens][heads][head_dim], all of one dtype, out the
 * same of either; lses: host array of device pointers, fp32 [batch][tokens][heads]; lse:
 * NULL, or the same. head_dim: 64 or 128. out and lse may be those of one of the parts (the
 * same view), but not overlap them otherwise. A part of lse -infinity is left out, whatever
 * its outputs hold; where all are, out is 0 and lse -infinity. A part's lse of NaN or
 * +infinity makes both NaN. Sums are held in fp32. Needs no plan. RC_ERR_UNSUPPORTED: another
 * head_dim, more than 2^20 heads, 2^34 rows (batch * tokens * heads) or more. */
rc_status_t rc_attn_join(hipStream_t stream, int parts, const rc_kv_view_t* outs, const float* const* lses,
                         int batch, int tokens, int heads, int head_dim, const rc_kv_view_t* out, float* lse);

#ifdef __cplusplus
}
#endif

#endif /* LIBRESCOMP_ATTN_H */
