/*
 * librescomp: an 8-bit key/value cache and the attention that reads it.
 *
 * A GPU of a sequence-parallel step attends from its own share of the tokens to
 * the keys and values of every peer, which reach it as reconstructions
 * (rc_decompress) or in full. It holds them here: blocks of 64 tokens, e4m3
 * codes with one power-of-two scale per block and key head, and one 8-bit mean
 * key per block and key head that a cheap score uses to choose blocks. Three
 * operators:
 *
 *   rc_kv_store    quantise new keys and values into the cache (whole sequences
 *                  or single tokens)
 *   rc_kv_attend   attention of new queries over the cache, or over chosen blocks
 *   rc_kv_select   choose the blocks that rc_kv_attend reads
 *
 * The conventions of librescomp.h hold: device pointers owned by the caller, 16-
 * byte aligned; calls are asynchronous on the given stream, never synchronise
 * the host and may be captured; calls on one plan are serialised on one stream;
 * a rejected request launches nothing and writes nothing.
 */
#ifndef LIBRESCOMP_KV_H
#define LIBRESCOMP_KV_H

#include "librescomp.h"

#ifdef __cplusplus
extern "C" {
#endif

#define RC_KV_BLOCK 64         /* tokens of a block                                  */
#define RC_KV_QTILE 128        /* the larger q_tile                                  */
#define RC_KV_MAX_BLOCKS 8192  /* blocks of one sequence (seq_blocks) at most        */

typedef struct rc_kv_plan* rc_kv_plan_t; /* opaque; owns its workspace only */

typedef struct {
  int32_t batch;       /* sequences of a call                                        */
  int32_t q_heads;     /* query heads, a multiple of kv_heads: query head h reads    */
  int32_t kv_heads;    /*   key head h / (q_heads / kv_heads)                        */
  int32_t head_dim;    /* 64 or 128                                                  */
  int32_t pool_blocks; /* blocks that the cache holds                                */
  int32_t seq_blocks;  /* blocks of one sequence at most (the table's row length)    */
} rc_kv_shape_t;

/* rc_kv_params_t.flags: query i of n sees the tokens up to its own, which is token
 * kv_len - n + i of its sequence (the queries are the last n tokens). Without it
 * every query sees all kv_len tokens. */
#define RC_KV_CAUSAL 1u

typedef struct {
  int32_t max_queries; /* query tokens of a sequence and call at most, >= 1          */
  float scale;         /* factor of the scores; 0: 1 / sqrt(head_dim)                */
  int32_t q_tile;      /* queries that share a choice of blocks: 1 or RC_KV_QTILE;   */
                       /*   0: the plan chooses none (rc_kv_select is refused)       */
  int32_t keep_blocks; /* blocks chosen per tile, 1..1024; 0 with q_tile 0. Causal   */
                       /*   tiles of RC_KV_QTILE need 3 (a tile's own positions may  */
                       /*   lie in 3 blocks, which are always chosen)                */
  uint32_t flags;      /* 0 or RC_KV_CAUSAL                                          */
} rc_kv_params_t;

/* The cache, all parts the caller's (D = head_dim, one [kv_heads] row per block):
 *   k            e4m3 codes [pool_blocks][kv_heads][D / 16][64 tokens][16]
 *   v            e4m3 codes [pool_blocks][kv_heads][4][D][16 tokens]
 *   k_scale      fp32 [pool_blocks][kv_heads], a power of two in 2^-40 .. 2^44;
 *   v_scale        a value is its code times its block's scale
 *   k_mean       int8 [pool_blocks][kv_heads][D]: the mean of the block's keys is
 *   k_mean_scale   about k_mean * k_mean_scale, fp32 [pool_blocks][kv_heads]
 * The orders inside a block are the ones in which the matrix units read it. */
typedef struct {
  void* k;
  void* v;
  float* k_scale;
  float* v_scale;
  int8_t* k_mean;
  float* k_mean_scale;
} rc_kv_cache_t;

/* Rows of head_dim contiguous values: element (b, t, h, d) of a tensor
 * [batch][tokens][heads][head_dim] is data[b * batch_stride + t * token_stride +
 * h * head_stride + d]. Strides are in elements, not negative, and keep every row
 * 16-byte aligned; an input's strides may be 0. An output's dimensions (those of more
 * than one) nest: in order of their strides, each stride passes what the dimensions
 * before it span, so no two rows overlap; any view of whole rows of a tensor does. A call
 * with no tokens or queries reads and writes nothing (data may be NULL) and returns RC_OK. */
typedef struct {
  void* data;
  rc_dtype_t dtype;
  int64_t batch_stride, token_stride, head_stride;
} rc_kv_view_t;

/* Validate the request and allocate the workspace (rc_kv_workspace_bytes) on the
 * current device. dtype: of the queries and outputs. Errors: RC_ERR_INVALID_ARG
 * (null pointer, bad value), RC_ERR_UNSUPPORTED (a valid value that this library
 * does not implement: another head_dim, more than RC_KV_MAX_BLOCKS blocks),
 * RC_ERR_HIP. */
rc_status_t rc_kv_plan_create(rc_kv_shape_t shape, rc_dtype_t dtype, const rc_kv_params_t* params,
                              rc_kv_plan_t* out);

/* Block tables. `table` is a device int32 [batch][seq_blocks]: block j of sequence
 * b is block table[b][j] of the pool; an entry outside the pool means that there is
 * no such block (nothing is stored to it, and its tokens are seen by no query).
 * NULL: block j of sequence b is block b * seq_blocks + j. Lengths and starts are
 * device int32 [batch]. */

/* Store `tokens` new tokens of every sequence, from position start[b] on. The
 * sequence then ends after them: what it held from start[b] on is gone. `count`
 * (device int32 [batch], or NULL): only the first count[b] of the new tokens are
 * there. k, v: [batch][tokens][kv_heads][head_dim], of either dtype.
 *   - A block's scale is the smallest power of two 2^e (e in -40..44) with
 *     max|x| <= 448 * 2^e over the block's finite values; codes are x / 2^e rounded
 *     to nearest even and clamped to +-448. NaN is stored as the NaN code 0xFF.
 *   - In a block that holds earlier tokens the scale never falls; if it rises, the
 *     earlier codes are rounded again in the new scale. Its slots after the new
 *     tokens keep what they hold. A block without earlier tokens is written whole,
 *     zero after the new tokens.
 *   - k_mean: T = sum of the block's key codes (NaN as 0; exact in fp32), a = max|T|: codes
 *     T * ((1 / a) * 127), rounded to nearest even, scale a / (127 * tokens) * 2^e,
 *     each operation rounded to fp32.
 * Tokens that fall outside [0, 64 * seq_blocks) are dropped; a negative start drops
 * the sequence's call. Sequences of one call must not share the blocks that they
 * write. */
rc_status_t rc_kv_store(rc_kv_plan_t plan, hipStream_t stream, const rc_kv_cache_t* cache,
                        const int32_t* table, const int32_t* start, const int32_t* count, int tokens,
                        const rc_kv_view_t* k, const rc_kv_view_t* v);

/* Choose blocks for `queries` query tokens (1..max_queries) of every sequence of
 * kv_len[b] tokens. q: [batch][queries][q_heads][head_dim] in the plan's dtype.
 *   score(query, head, block) = (float(qc . k_mean) * k_mean_scale) * max|q|, where
 *   qc = q * ((1 / max|q|) * 127), rounded to nearest even, in 8 bits (each
 *   operation rounded to fp32; where the factor is not finite, for rows of zeros and of
 *   less than 2^-121, qc is 0; the products of qc and k_mean are whole numbers and
 *   their sum is exact, so the choice does not depend on the order of a sum).
 * The score of a block for a tile is the largest over the tile's queries that see
 * its first token and over the query heads of the key head. The keep_blocks blocks
 * of the highest score are chosen, ties to the lower index; with RC_KV_CAUSAL the
 * blocks of the tile's own positions come first. Every block that is there and that a
 * query of the tile sees can be chosen: a score that is NaN (a query that holds an
 * infinity has no other) counts as -infinity, and that is the lowest score. A NaN in a
 * query counts as 0 here. blocks: device int32 [batch][kv_heads][ceil(queries / q_tile)]
 * [keep_blocks], ascending, -1 after the last.
 * max_len: a bound of kv_len that the host knows (0: 64 * seq_blocks). Longer
 * lengths are cut to it, and to 64 * seq_blocks; negative ones count as 0. */
rc_status_t rc_kv_select(rc_kv_plan_t plan, hipStream_t stream, const rc_kv_cache_t* cache,
                         const int32_t* table, const int32_t* kv_len, int64_t max_len, int queries,
                         const rc_kv_view_t* q, int32_t* blocks);

/* Attention: out = softmax(scale * q k^T) v over the tokens that each query sees
 * and, with `blocks` (as rc_kv_select lays them out; NULL: all), that lie in the
 * blocks chosen for its tile. A list ends at its first entry that is negative or not
 * below the number of blocks that the tile sees; entries may be in any order, and the
 * same block twice counts twice.
 * out: [batch][queries][q_heads][head_dim] in the plan's dtype.
 * lse (NULL, or fp32 [batch][queries][q_heads]): the natural logarithm of the sum
 * of the exponentials, to join this result with attention over other tokens. A
 * query that sees no token, or whose scores are all -infinity, gets 0 and -infinity.
 * Precision: sums, the running maximum and outputs are held in fp32 and rounded once.
 * With bf16 outputs the weights are rounded to f16 (11 bits) for their product with v, not
 * for their sum: before the rounding to bf16 an output is within about 2^-11 of the
 * weighted mean of |v|. In fp32, queries and weights are sums of two f16 (22 bits). Values
 * of a query under 2^-29 of its largest lose bits.
 * NaN: a key's makes the outputs and the lse of the queries that see it NaN; a query's,
 * or scores of +infinity, its own. A value's reaches the outputs, not the lse, of the
 * queries that see it and, with RC_KV_CAUSAL, may reach the outputs of earlier queries of
 * the call for which its block is read (its weight there is zero, and zero times NaN is
 * NaN). What a block holds after its sequence's end reaches no one. */
rc_status_t rc_kv_attend(rc_kv_plan_t plan, hipStream_t stream, const rc_kv_cache_t* cache,
                         const int32_t* table, const int32_t* kv_len, int64_t max_len, int queries,
                         const rc_kv_view_t* q, const int32_t* blocks, const rc_kv_view_t* out, float* lse);

/* Free the plan and its workspace; no launched work may still use it. NULL is
 * accepted. */
rc_status_t rc_kv_plan_destroy(rc_kv_plan_t plan);

/* Device workspace that the plan owns. 0 for a NULL plan. */
size_t rc_kv_workspace_bytes(rc_kv_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* LIBRESCOMP_KV_H */
