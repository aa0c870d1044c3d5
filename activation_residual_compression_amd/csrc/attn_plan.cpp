// Host side of attention over packed sequences: validation, workspace, choice of the
// kernel and of the split over the keys. And of the join, which needs no plan.
#include "../../include/librescomp_attn.h"

#include <float.h>
#include <math.h>
#include <stdlib.h>

#include <algorithm>
#include <new>

#include "attn.hpp"
#include "views.hpp"

struct rc_attn_plan {
  rc_attn_shape_t shape;
  rc_dtype_t dtype;
  rc_attn_params_t params;
  void* ws = nullptr;  // partial results: outputs, (m, l); then the counters
  size_t ws_bytes = 0;
  int64_t part_rows = 0;        // rows of partial results that it holds
  uint32_t* arrived = nullptr;  // [kFewGroups]
};

namespace {

using rc::at4;
using rc::ceil_div;
using rc::rows_of;

// Groups of rows that may have several parts, at most.
constexpr int64_t kFewGroups = 1536;

struct Way {
  int splits, chunk;
  int64_t part_rows;  // rows of partial results; 0 with one part
};

Way way_of(const rc_attn_plan* pl, int64_t seqs, int64_t q_tokens, int64_t kv_tokens, int64_t max_q, int64_t max_kv,
           int64_t most_rows) {
  const rc_attn_shape_t& s = pl->shape;
  const int64_t group = s.q_heads / s.kv_heads, rows = q_tokens * s.q_heads;
  const int64_t groups = ceil_div(max_q * group, 16), base = seqs * s.kv_heads * groups;
  // Blocks of threads that the CUs hold at once.
  const int64_t at_once = 256 * (pl->dtype == RC_F32 ? 2 : 3);
  Way w{1, (int)std::max<int64_t>(max_kv, 1), 0};
  if (base > kFewGroups || rows == 0 || (pl->dtype == RC_BF16 && max_q * group > 64)) return w;
  // equal parts of all keys that are read, one for each block of threads
  const int64_t read = kv_tokens * s.kv_heads * groups;
  const int64_t chunk = std::max<int64_t>(256, ceil_div(ceil_div(read, at_once), 64) * 64);
  const int64_t splits = std::min({ceil_div(max_kv, chunk), most_rows / rows, (int64_t)256});
  if (splits <= 1) return w;
  w.splits = (int)splits;
  w.chunk = (int)std::max(chunk, ceil_div(ceil_div(max_kv, splits), 64) * 64);
  w.part_rows = splits * rows;
  return w;
}

size_t part_bytes(const rc_attn_plan* pl, int64_t part_rows) {
  return (size_t)part_rows * ((size_t)pl->shape.head_dim * 4 + sizeof(float2));
}

// Rows of partial results that the workspace is made for: what calls of one sequence, of
// all, and of powers of two between need, with few and with all queries, at most half a
// gigabyte. A call that would need more takes fewer parts.
int64_t part_rows_at_most(const rc_attn_plan* pl) {
  const rc_attn_shape_t& s = pl->shape;
  const int64_t cap = ((int64_t)512 << 20) / (int64_t)part_bytes(pl, 1);
  int64_t most = 0;
  for (int64_t n = 1;; n = std::min<int64_t>(2 * n, s.max_seqs)) {
    for (int64_t q = 1;; q = std::min<int64_t>(2 * q, s.max_queries)) {
      if (q >= n) most = std::max(most, way_of(pl, n, q, s.max_keys, ceil_div(q, n), s.max_keys, cap).part_rows);
      if (q == s.max_queries) break;
    }
    if (n == s.max_seqs) return most;
  }
}

rc_status_t check(const rc_attn_shape_t& s, rc_dtype_t dtype, const rc_attn_params_t* p) {
  if (!p) return RC_ERR_INVALID_ARG;
  if (s.q_heads < 1 || s.kv_heads < 1 || s.head_dim < 1 || s.max_seqs < 1 || s.max_queries < 1 || s.max_keys < 1)
    return RC_ERR_INVALID_ARG;
  if (s.q_heads % s.kv_heads) return RC_ERR_INVALID_ARG;
  if (dtype != RC_BF16 && dtype != RC_F32) return RC_ERR_INVALID_ARG;
  if (!(p->scale >= 0.0f) || !isfinite(p->scale) || p->flags & ~RC_ATTN_CAUSAL) return RC_ERR_INVALID_ARG;
  if (s.head_dim != 64 && s.head_dim != 128) return RC_ERR_UNSUPPORTED;
  if (s.max_seqs > 65535 || s.kv_heads > 32767) return RC_ERR_UNSUPPORTED;
  if (s.max_keys > 1 << 30 || (int64_t)s.max_queries * s.q_heads >= (int64_t)1 << 30) return RC_ERR_UNSUPPORTED;
  return RC_OK;
}

}  // namespace

extern "C" {

rc_status_t rc_attn_plan_create(rc_attn_shape_t shape, rc_dtype_t dtype, const rc_attn_params_t* params,
                                rc_attn_plan_t* out) {
  if (!out) return RC_ERR_INVALID_ARG;
  *out = nullptr;
  const rc_status_t st = check(shape, dtype, params);
  if (st != RC_OK) return st;
  rc_attn_plan* pl = new (std::nothrow) rc_attn_plan;
  if (!pl) return RC_ERR_HIP;
  pl->shape = shape;
  pl->dtype = dtype;
  pl->params = *params;
  pl->part_rows = part_rows_at_most(pl);
  if (pl->part_rows) {
    const size_t parts = part_bytes(pl, pl->part_rows), counts = kFewGroups * sizeof(uint32_t);
    if (hipMalloc(&pl->ws, parts + counts) != hipSuccess) {
      delete pl;
      return RC_ERR_HIP;
    }
    pl->ws_bytes = parts + counts;
    pl->arrived = reinterpret_cast<uint32_t*>(static_cast<char*>(pl->ws) + parts);
    // done before the first call, which may be on a stream that does not wait for this one
    if (hipMemset(pl->arrived, 0, counts) != hipSuccess || hipStreamSynchronize(nullptr) != hipSuccess) {
      (void)hipFree(pl->ws);
      delete pl;
      return RC_ERR_HIP;
    }
  }
  *out = pl;
  return RC_OK;
}

rc_status_t rc_attn_packed(rc_attn_plan_t pl, hipStream_t stream, int seqs, const int32_t* q_offsets,
                           const int32_t* kv_offsets, int q_tokens, int kv_tokens, int max_q, int max_kv,
                           const rc_kv_view_t* q, const rc_kv_view_t* k, const rc_kv_view_t* v,
                           const rc_kv_view_t* out, float* lse) {
  if (!pl || !q_offsets) return RC_ERR_INVALID_ARG;
  const rc_attn_shape_t& s = pl->shape;
  if (seqs < 0 || seqs > s.max_seqs || q_tokens < 0 || q_tokens > s.max_queries || kv_tokens < 0 ||
      kv_tokens > s.max_keys || max_q < 0 || max_kv < 0)
    return RC_ERR_INVALID_ARG;
  if (!at4(q_offsets) || (kv_offsets && !at4(kv_offsets)) || (lse && !at4(lse))) return RC_ERR_ALIGNMENT;
  rc::AttnArgs a;
  rc_status_t st = rows_of(q, 1, q_tokens, s.q_heads, s.head_dim, false, &a.q);
  if (st == RC_OK) st = rows_of(k, 1, kv_tokens, s.kv_heads, s.head_dim, false, &a.k);
  if (st == RC_OK) st = rows_of(v, 1, kv_tokens, s.kv_heads, s.head_dim, false, &a.v);
  if (st == RC_OK) st = rows_of(out, 1, q_tokens, s.q_heads, s.head_dim, true, &a.out);
  if (st != RC_OK) return st;
  if (q->dtype != pl->dtype || k->dtype != pl->dtype || v->dtype != pl->dtype || out->dtype != pl->dtype)
    return RC_ERR_INVALID_ARG;
  if (seqs == 0 || q_tokens == 0) return RC_OK;
  a.lse = lse;
  a.q_off = q_offsets;
  a.kv_off = kv_offsets ? kv_offsets : q_offsets;
  a.seqs = seqs;
  a.q_tokens = q_tokens;
  a.kv_tokens = kv_tokens;
  a.max_q = max_q ? std::min(max_q, q_tokens) : q_tokens;
  a.max_kv = max_kv ? std::min(max_kv, kv_tokens) : kv_tokens;
  a.q_heads = s.q_heads;
  a.kv_heads = s.kv_heads;
  a.group = s.q_heads / s.kv_heads;
  a.dim = s.head_dim;
  a.causal = (pl->params.flags & RC_ATTN_CAUSAL) != 0;
  constexpr float kLog2e = 1.44269504088896340736f;
  a.scale = fminf((pl->params.scale > 0.0f ? pl->params.scale : 1.0f / sqrtf((float)s.head_dim)) * kLog2e, FLT_MAX);
  const Way w = way_of(pl, seqs, q_tokens, kv_tokens, a.max_q, a.max_kv, pl->part_rows);
  a.splits = w.splits;
  a.chunk = w.chunk;
  a.part = static_cast<float*>(pl->ws);
  a.part_ml = reinterpret_cast<float2*>(a.part + w.part_rows * s.head_dim);
  a.arrived = pl->arrived;
  const int64_t rows = (int64_t)a.max_q * a.group;
  if (pl->dtype == RC_BF16 && rows > 16 && w.splits == 1) {
    const char* e = getenv("RC_U");
    const int u = e ? atoi(e) : (int64_t)q_tokens * a.group / 256 * a.kv_heads >= 200 ? 2 : 1;
    return rc::launch_attn_many(a, u, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
  }
  return rc::launch_attn_few(a, pl->dtype == RC_BF16, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
}

rc_status_t rc_attn_plan_destroy(rc_attn_plan_t pl) {
  if (!pl) return RC_OK;
  hipError_t err = hipSuccess;
  if (pl->ws) err = hipFree(pl->ws);
  delete pl;
  return err == hipSuccess ? RC_OK : RC_ERR_HIP;
}

size_t rc_attn_workspace_bytes(rc_attn_plan_t pl) { return pl ? pl->ws_bytes : 0; }

rc_status_t rc_attn_join(hipStream_t stream, int parts, const rc_kv_view_t* outs, const float* const* lses,
                         int batch, int tokens, int heads, int head_dim, const rc_kv_view_t* out, float* lse) {
  if (parts < 1 || parts > RC_ATTN_MAX_PARTS || !outs || !lses || batch < 0 || tokens < 0 || heads < 0 || head_dim < 1)
    return RC_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return RC_ERR_UNSUPPORTED;
  rc::AttnJoinArgs a;
  const int64_t rows = (int64_t)batch * tokens * std::min<int64_t>(heads, 1 << 20);
  for (int i = 0; i < parts; ++i) {
    const rc_status_t st = rows_of(&outs[i], batch, rows ? tokens : 0, heads, head_dim, false, &a.in[i]);
    if (st != RC_OK) return st;
    if (outs[i].dtype != outs[0].dtype || (rows && !lses[i])) return RC_ERR_INVALID_ARG;
    if (!at4(lses[i])) return RC_ERR_ALIGNMENT;
    a.lses[i] = lses[i];
  }
  const rc_status_t st = rows_of(out, batch, rows ? tokens : 0, heads, head_dim, true, &a.out);
  if (st != RC_OK) return st;
  if (lse && !at4(lse)) return RC_ERR_ALIGNMENT;
  if (heads > 1 << 20 || rows >= (int64_t)1 << 34) return RC_ERR_UNSUPPORTED;
  if (rows == 0) return RC_OK;
  a.lse = lse;
  a.parts = parts;
  a.tokens = tokens;
  a.heads = heads;
  a.dim = head_dim;
  a.rows = rows;
  return rc::launch_attn_join(a, outs[0].dtype == RC_BF16, out->dtype == RC_BF16, stream) == hipSuccess ? RC_OK
                                                                                                       : RC_ERR_HIP;
}

}  // extern "C"
