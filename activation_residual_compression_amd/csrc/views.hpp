// Host side: checks of arguments that the key/value cache, packed attention and the
// cache's pages share.
#pragma once

#include <algorithm>

#include "kv.hpp"
#include "memory.hpp"

namespace rc {

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

inline bool at16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
inline bool at4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

inline rc_status_t check_cache(const rc_kv_cache_t* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->k_mean || !c->k_mean_scale) return RC_ERR_INVALID_ARG;
  if (!at16(c->k) || !at16(c->v) || !at16(c->k_scale) || !at16(c->v_scale) || !at16(c->k_mean) ||
      !at16(c->k_mean_scale))
    return RC_ERR_ALIGNMENT;
  return RC_OK;
}

// A view of [batch][tokens][heads][dim]; strides of dimensions of size 1 do not count. The
// rows of an output must not overlap: in order of their strides, each dimension's passes
// what those before it span.
inline rc_status_t rows_of(const rc_kv_view_t* v, int64_t batch, int64_t tokens, int64_t heads, int64_t dim,
                           bool out, KvRows* r) {
  if (!v || (!v->data && tokens > 0)) return RC_ERR_INVALID_ARG;
  if (v->dtype != RC_BF16 && v->dtype != RC_F32) return RC_ERR_INVALID_ARG;
  if (!at16(v->data)) return RC_ERR_ALIGNMENT;
  const int64_t unit = v->dtype == RC_BF16 ? 8 : 4, n[3] = {batch, tokens, heads};
  int64_t st[3] = {v->batch_stride, v->token_stride, v->head_stride};
  for (int i = 0; i < 3; ++i) {
    if (n[i] <= 1) st[i] = 0;
    else if (st[i] < (out ? dim : 0) || st[i] >= (int64_t)1 << 40) return RC_ERR_INVALID_ARG;
    if (st[i] % unit) return RC_ERR_ALIGNMENT;
  }
  if (out) {
    int order[3] = {0, 1, 2};
    std::sort(order, order + 3, [&](int x, int y) { return st[x] < st[y]; });
    __int128 span = dim;
    for (int i : order) {
      if (n[i] <= 1) continue;
      if (st[i] < span) return RC_ERR_INVALID_ARG;
      span += (__int128)st[i] * (n[i] - 1);
    }
  }
  *r = {v->data, st[0], st[1], st[2]};
  return RC_OK;
}

}  // namespace rc
