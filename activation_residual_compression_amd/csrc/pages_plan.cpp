// Host side of the cache's pages: validation and workspace.
#include "../../include/librescomp_pages.h"

#include <new>

#include "pages.hpp"
#include "views.hpp"

struct rc_pages_plan {
  rc_pages_shape_t shape;
  rc::PageGeom geom;
  rc::PageWork work;
  void* ws = nullptr;
  size_t ws_bytes = 0;
};

namespace {

using rc::at4;

rc_status_t check(const rc_pages_shape_t& s) {
  if (s.slots < 1 || s.kv_heads < 1 || s.head_dim < 1 || s.pool_blocks < 1 || s.seq_blocks < 1) return RC_ERR_INVALID_ARG;
  if (s.head_dim != 64 && s.head_dim != 128) return RC_ERR_UNSUPPORTED;
  if (s.slots > 65535 || s.kv_heads > 32767 || s.seq_blocks > RC_KV_MAX_BLOCKS) return RC_ERR_UNSUPPORTED;
  if ((int64_t)s.slots * s.seq_blocks >= (int64_t)1 << 31 || s.pool_blocks > 1 << 28) return RC_ERR_UNSUPPORTED;
  return RC_OK;
}

// The workspace's arrays from `base` on (null: sizes only); returns the bytes.
size_t carve(rc_pages_plan* pl, char* base) {
  const rc_pages_shape_t& s = pl->shape;
  size_t at = 0;
  const auto take = [&](auto*& p, size_t n) {
    p = reinterpret_cast<std::remove_reference_t<decltype(p)>>(base + at);
    at += (n * sizeof(*p) + 63) / 64 * 64;
  };
  const size_t pool = (size_t)s.pool_blocks;
  rc::PageWork& w = pl->work;
  take(w.writers, pool);
  take(w.first, pool);
  take(w.list, pool);
  take(w.old, pool);
  take(w.place, pool);
  take(w.pairs, (size_t)s.slots);
  take(w.count, 1);
  take(w.rows, (size_t)s.slots * (size_t)s.seq_blocks);
  return at;
}

rc::PageParts parts_of(const rc_kv_cache_t* c) {
  return {{(char*)c->k, (char*)c->v, (char*)c->k_mean, (char*)c->k_scale, (char*)c->v_scale, (char*)c->k_mean_scale}};
}

// State that every call but copy takes, and int32 arrays that it needs or may have.
rc_status_t check_ints(const int32_t* const* needed, int n, const int32_t* x = nullptr, const int32_t* y = nullptr) {
  for (int i = 0; i < n; ++i)
    if (!needed[i]) return RC_ERR_INVALID_ARG;
  for (int i = 0; i < n; ++i)
    if (!at4(needed[i])) return RC_ERR_ALIGNMENT;
  return at4(x) && at4(y) ? RC_OK : RC_ERR_ALIGNMENT;
}

rc_status_t status_of(hipError_t err) { return err == hipSuccess ? RC_OK : RC_ERR_HIP; }

}  // namespace

extern "C" {

rc_status_t rc_pages_plan_create(rc_pages_shape_t shape, rc_pages_plan_t* out) {
  if (!out) return RC_ERR_INVALID_ARG;
  *out = nullptr;
  const rc_status_t st = check(shape);
  if (st != RC_OK) return st;
  rc_pages_plan* pl = new (std::nothrow) rc_pages_plan;
  if (!pl) return RC_ERR_HIP;
  pl->shape = shape;
  const int h = shape.kv_heads, d = shape.head_dim;
  pl->geom = {shape.slots, shape.pool_blocks, shape.seq_blocks, {h * RC_KV_BLOCK * d, h * RC_KV_BLOCK * d, h * d, 4 * h, 4 * h, 4 * h}};
  pl->ws_bytes = carve(pl, nullptr);
  const size_t pool = (size_t)shape.pool_blocks;
  // done before the first call, which may be on a stream that does not wait for this one
  if (!rc::allocate(&pl->ws, pl->ws_bytes)) {
    delete pl;
    return RC_ERR_HIP;
  }
  carve(pl, static_cast<char*>(pl->ws));
  if (hipMemset(pl->work.writers, 0, pool * 4) != hipSuccess || hipMemsetD32(pl->work.first, INT32_MAX, pool) != hipSuccess ||
      hipStreamSynchronize(nullptr) != hipSuccess) {
    (void)hipFree(pl->ws);
    delete pl;
    return RC_ERR_HIP;
  }
  *out = pl;
  return RC_OK;
}

rc_status_t rc_pages_reserve(rc_pages_plan_t pl, hipStream_t stream, const rc_kv_cache_t* cache, int32_t* refs,
                             int32_t* table, const int32_t* start, const int32_t* tokens, int32_t* missing) {
  if (!pl) return RC_ERR_INVALID_ARG;
  const int32_t* const needed[] = {refs, table, start, tokens};
  rc_status_t st = check_ints(needed, 4, missing);
  if (st == RC_OK) st = rc::check_cache(cache);
  if (st != RC_OK) return st;
  return status_of(rc::launch_pages_reserve(pl->geom, pl->work, parts_of(cache), refs, table, start, tokens, missing, stream));
}

rc_status_t rc_pages_fork(rc_pages_plan_t pl, hipStream_t stream, int32_t* refs, int32_t* table,
                          const int32_t* source, const int32_t* length) {
  if (!pl) return RC_ERR_INVALID_ARG;
  const int32_t* const needed[] = {refs, table, source, length};
  const rc_status_t st = check_ints(needed, 4);
  if (st != RC_OK) return st;
  return status_of(rc::launch_pages_fork(pl->geom, pl->work, refs, table, source, length, stream));
}

rc_status_t rc_pages_free(rc_pages_plan_t pl, hipStream_t stream, int32_t* refs, int32_t* table, const int32_t* keep) {
  if (!pl) return RC_ERR_INVALID_ARG;
  const int32_t* const needed[] = {refs, table, keep};
  const rc_status_t st = check_ints(needed, 3);
  if (st != RC_OK) return st;
  return status_of(rc::launch_pages_free(pl->geom, refs, table, keep, stream));
}

rc_status_t rc_pages_compact(rc_pages_plan_t pl, hipStream_t stream, const rc_kv_cache_t* cache, int32_t* refs,
                             int32_t* table, int32_t* used, int32_t* moved) {
  if (!pl) return RC_ERR_INVALID_ARG;
  const int32_t* const needed[] = {refs, table};
  rc_status_t st = check_ints(needed, 2, used, moved);
  if (st == RC_OK) st = rc::check_cache(cache);
  if (st != RC_OK) return st;
  return status_of(rc::launch_pages_compact(pl->geom, pl->work, parts_of(cache), refs, table, used, moved, stream));
}

rc_status_t rc_pages_copy(rc_pages_plan_t pl, hipStream_t stream, const rc_kv_cache_t* from,
                          const rc_kv_cache_t* to, const int32_t* src, const int32_t* dst, int count) {
  if (!pl || count < 0) return RC_ERR_INVALID_ARG;
  rc_status_t st = rc::check_cache(from);
  if (st == RC_OK) st = rc::check_cache(to);
  if (st != RC_OK) return st;
  if (count == 0) return RC_OK;
  const int32_t* const needed[] = {src, dst};
  st = check_ints(needed, 2);
  if (st != RC_OK) return st;
  return status_of(rc::launch_pages_copy(pl->geom, parts_of(from), parts_of(to), src, dst, count, stream));
}

rc_status_t rc_pages_plan_destroy(rc_pages_plan_t pl) {
  if (!pl) return RC_OK;
  const hipError_t err = hipFree(pl->ws);
  delete pl;
  return status_of(err);
}

size_t rc_pages_workspace_bytes(rc_pages_plan_t pl) { return pl ? pl->ws_bytes : 0; }

}  // extern "C"
