/*
 * librescomp: the pages of a key/value cache. Sequences of the cache of
 * librescomp_kv.h take their blocks from a common pool through a table; here the
 * blocks are given out, shared, copied, given back and moved together, all on the
 * device and in stream order, with results that do not depend on timing:
 *
 *   rc_pages_reserve   give sequences blocks of their own for new tokens
 *   rc_pages_fork      let sequences continue others (shared blocks, copied when written)
 *   rc_pages_free      give back blocks: whole sequences, or their last tokens
 *   rc_pages_compact   move the blocks in use to the front of the pool
 *   rc_pages_copy      copy blocks, inside a cache or to another one
 *
 * State, all the caller's:
 *   table   device int32 [slots][seq_blocks], a row for each sequence that the cache can
 *           hold: entry j of row s is the pool block of its tokens 64 j .. 64 j + 63. An
 *           entry outside the pool means that there is no such block.
 *   refs    device int32 [pool_blocks]: how often a block stands in the table. Blocks of
 *           0 (or less) are free. A caller that counts itself among a block's holders
 *           keeps it from being given out. An empty cache: table all -1, refs all 0.
 * rc_kv_store writes the blocks that a row names: before it does, rc_pages_reserve makes
 * sure that there are such, and that no other sequence reads them.
 *
 * The conventions of librescomp_kv.h hold: device pointers owned by the caller; calls are
 * asynchronous on the given stream, never synchronise the host and may be captured; calls
 * on one plan, table or cache are serialised on one stream; a rejected request launches
 * nothing and writes nothing.
 */
#ifndef LIBRESCOMP_PAGES_H
#define LIBRESCOMP_PAGES_H

#include "librescomp_kv.h"

#ifdef __cplusplus
extern "C" {
#endif

typedef struct rc_pages_plan* rc_pages_plan_t; /* opaque; owns its workspace only */

typedef struct {
  int32_t slots;       /* rows of the table, at most 65535                           */
  int32_t kv_heads;    /* of the cache, at most 32767                                */
  int32_t head_dim;    /* 64 or 128                                                  */
  int32_t pool_blocks; /* blocks that the cache holds                                */
  int32_t seq_blocks;  /* blocks of one sequence at most (the table's row length)    */
} rc_pages_shape_t;

/* Validate the request and allocate the workspace (rc_pages_workspace_bytes) on the
 * current device. Errors: RC_ERR_INVALID_ARG (null pointer, bad value),
 * RC_ERR_UNSUPPORTED (a valid value that this library does not implement: another
 * head_dim, more than RC_KV_MAX_BLOCKS blocks of a sequence), RC_ERR_HIP. */
rc_status_t rc_pages_plan_create(rc_pages_shape_t shape, rc_pages_plan_t* out);

/* Make room for tokens[s] new tokens of every sequence s from position start[s] on
 * (device int32 [slots]; no tokens, or a negative start: nothing for s). Of the entries of
 * its row that they fall into (those past the row's end: none),
 *   - one that has no block gets a free one;
 *   - one whose block others hold too (refs > 1) gets a free one in its place. If it
 *     holds tokens before start[s], its contents are copied. If every holder of a block
 *     is such an entry of this call, the first of them (by s, then by position) keeps it.
 * Free blocks are given out in ascending order, by s, then by position; refs follow.
 * All or nothing: if fewer blocks are free than the call needs, nothing changes. missing
 * (NULL, or device int32 [1]): how many are lacking, 0 if it was done. */
rc_status_t rc_pages_reserve(rc_pages_plan_t plan, hipStream_t stream, const rc_kv_cache_t* cache, int32_t* refs,
                             int32_t* table, const int32_t* start, const int32_t* tokens, int32_t* missing);

/* Sequence s becomes a continuation of sequence source[s] of length[s] tokens (device
 * int32 [slots]): its row is replaced by the first ceil(length[s] / 64) entries of the
 * other, and refs follow (blocks that nobody holds any more are free). All rows are read as
 * they were before the call, so sequences may be exchanged or follow one another.
 * source[s] outside 0 .. slots - 1: nothing for s; source[s] = s: cut to length[s].
 * Nothing is copied: the block that both go on writing is, by rc_pages_reserve. */
rc_status_t rc_pages_fork(rc_pages_plan_t plan, hipStream_t stream, int32_t* refs, int32_t* table,
                          const int32_t* source, const int32_t* length);

/* Keep the first keep[s] tokens (device int32 [slots]; negative: none) of every sequence:
 * the entries behind them become -1, and refs follow. */
rc_status_t rc_pages_free(rc_pages_plan_t plan, hipStream_t stream, int32_t* refs, int32_t* table,
                          const int32_t* keep);

/* Move the U blocks in use (refs > 0) to pool places 0 .. U - 1: the i-th one in use at or
 * after U goes to the i-th free place before U, contents, refs and entries of the table; the
 * others stay. used (NULL, or device int32 [1]): U. moved (NULL, or device int32
 * [pool_blocks]): for each block its place now, -1 for a free one. Places from U on keep
 * the contents that they had. */
rc_status_t rc_pages_compact(rc_pages_plan_t plan, hipStream_t stream, const rc_kv_cache_t* cache, int32_t* refs,
                             int32_t* table, int32_t* used, int32_t* moved);

/* Copy the contents of block src[i] of `from` to block dst[i] of `to` for i < count (device
 * int32 [count]; pairs with an index outside the pool: nothing). Both caches are of the
 * plan's geometry and the same or apart in memory. A place is the destination of one pair
 * at most; in one cache, a destination is not a source too, but for src[i] = dst[i]. */
rc_status_t rc_pages_copy(rc_pages_plan_t plan, hipStream_t stream, const rc_kv_cache_t* from,
                          const rc_kv_cache_t* to, const int32_t* src, const int32_t* dst, int count);

/* Free the plan and its workspace; no launched work may still use it. NULL is
 * accepted. */
rc_status_t rc_pages_plan_destroy(rc_pages_plan_t plan);

/* Device workspace that the plan owns. 0 for a NULL plan. */
size_t rc_pages_workspace_bytes(rc_pages_plan_t plan);

#ifdef __cplusplus
}
#endif

#endif /* LIBRESCOMP_PAGES_H */
