// Host side of the key/value cache: validation, workspace, choice of the kernel
// and of the split over the keys.
#include <math.h>

#include <algorithm>
#include <new>

#include "../../include/librescomp_kv.h"
#include "kv.hpp"

struct rc_kv_plan {
  rc_kv_shape_t shape;
  rc_dtype_t dtype;
  rc_kv_params_t params;
  void* ws = nullptr;  // partial results: outputs, (m, l), numbers of parts
  size_t ws_bytes = 0;
  int64_t part_rows = 0;  // rows of partial results that it holds
  uint32_t* arrived = nullptr;  // [kFewGroups], after them
};

namespace {

int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Groups of rows of the kernel for few rows that may have several parts, at most.
constexpr int64_t kFewGroups = 1536;

// How a call runs: which kernel, and in how many parts of which length a group of
// rows reads its blocks.
struct Way {
  bool few;
  int splits, chunk;
  int64_t part_rows;  // rows of partial results; 0 with one part
};

Way way_of(const rc_kv_plan* pl, int64_t queries, int64_t blocks, bool chosen, int64_t most_rows) {
  const rc_kv_shape_t& s = pl->shape;
  const int64_t group = s.q_heads / s.kv_heads, rows = queries * group;
  const bool own_lists = chosen && pl->params.q_tile == 1;
  Way w;
  const int64_t heads = (int64_t)s.batch * s.kv_heads;
  int64_t splits = 1;
  blocks = std::max<int64_t>(blocks, 1);
  // Up to 64 rows, the kernel for few reads (and converts) K and V once more for each
  // 16 rows after the first, and the kernel for many has a larger tile than rows and a
  // second launch for the join. Measured in us, few and many, bf16, 8 key heads of 128,
  // rows 32 and 64: one sequence of 2000 tokens (4 MB) 12 and 17, 12 and 17; 32 of 4096
  // (268 MB) 97 and 72, 175 and 81: equal at about 45 and 12 MB. In fp32 with 64
  // channels, where the tile is 64 rows of twice the products, 32 rows over 134 MB are
  // 44 and 61, and 48 rows 65 and 67.
  const int64_t again = (ceil_div(std::min<int64_t>(rows, 64), 16) - 1) * heads * blocks * 128 * s.head_dim;
  w.few = own_lists || rows <= 16 ||
          (rows <= 64 && (again <= (int64_t)32 << 20 || (rows <= 32 && s.head_dim == 64 && pl->dtype == RC_F32)));
  if (w.few) {
    const int64_t base = heads * (own_lists ? queries * ceil_div(group, 16) : ceil_div(rows, 16));
    // The time in microseconds: the bytes at 5.8 TB/s, or the waves' blocks one after
    // the other (2.4 each) where that is longer; 4 for the start and end of a round of
    // the blocks of threads that the CUs hold at once; for the join 5, and 0.4 for each
    // part. Measured: 32 sequences of 8192 tokens, 8 key heads of 128, 94 us in one part
    // and 98, 101, 107, 109 in 2, 3, 4, 6; 4 of 65536 tokens 97 us in 7 parts, 113 in 4, 109
    // in 24, 118 in 32; 8 of 32 chosen blocks 11.3 us in 4, 12.5 in 2, 12.9 in 8.
    const int64_t at_once = 256 * (s.head_dim == 128 ? (pl->dtype == RC_F32 ? 2 : 3) : 4);
    const int64_t most = base <= kFewGroups ? std::min({ceil_div(blocks, 4), most_rows / (heads * rows), (int64_t)256}) : 1;
    const double read_us = (double)base * (double)blocks * (128.0 * s.head_dim) / 5.8e6;
    double best = 0.0;
    for (int64_t p = 1; p <= std::max<int64_t>(most, 1); ++p) {
      const double rounds = (double)ceil_div(base * p, at_once), steps = (double)ceil_div(ceil_div(blocks, p), 4);
      const double cost = std::max(read_us, rounds * steps * 2.4) + 4.0 * rounds + (p > 1 ? 5.0 + 0.4 * (double)p : 0.0);
      if (p == 1 || cost < best) {
        best = cost;
        splits = p;
      }
    }
  } else {
    // Blocks of threads that the CUs run at full rate, two each, and rows of each (the
    // kernel's). Three of the four forms fit a third, but then each takes longer a step:
    // planned with 768 the video share takes 713 us and not 698, fp32 image share 151 and
    // 141, 1111 queries over 8888 in fp32, 30 heads of 64, 210 and 182; a few calls gain
    // (3000 over 3000, 16 heads of 64 on 2, 48 and 64).
    const int64_t at_once = 512, tile = s.head_dim == 128 && pl->dtype == RC_F32 ? 32 : 64;
    const int64_t base = heads * ceil_div(rows, tile);
    // The time in steps of four blocks, one a wave (about 3.6 us where the CUs are full),
    // and one more for the start and end of a block of threads: whole rounds of equal
    // parts, or for causal rows, whose parts differ and are started longest first, the
    // average and half the longest. Partial results cost a write and a read, and the
    // launch that joins them 1.5 steps. Measured in us, as it is and with one weight
    // changed, over 30 calls, the ones that change most:
    //   start and end 1   at 0: video share 699 and 718, fp32 2222 over 8000, 16 / 4 heads of
    //                     128, 290 and 304, 500 over 5000, 24 heads, 80 and 77; at 3: causal
    //                     512 over 8000, 24 heads of 128, 66 and 76, 3000 over 3000 64 and 48
    //   longest part 0.5  at 0: causal 512 over 8000 66 and 76, 1000 over 1000, 12 heads of
    //                     64, 17.0 and 13.5; at 1: causal 2000 over 4000, 2 x 12 heads of 64,
    //                     55 and 64, fp32 4444 over 8888 472 and 488
    //   write and read    at 0: video share 699 and 720, chosen blocks of it 194 and 213,
    //                     causal 4000 over 4000, 16 / 4 heads of 128, 77 and 112
    //   launch 1.5        at 0: none; at 4: 3000 over 3000 64 and 48, 1000 over 1000 17.0 and 13.4
    const bool causal = (pl->params.flags & RC_KV_CAUSAL) && !chosen;
    double best = 0.0;
    for (int64_t p = 1; p <= std::min({(int64_t)16, ceil_div(blocks, 8), std::max<int64_t>(most_rows / (heads * rows), 1)});
         ++p) {
      const double len = (double)ceil_div(ceil_div(blocks, p), 4) + 1.0;
      const double mean = (causal ? std::max(1.0, 0.25 * ((double)blocks - (double)std::min(queries / 128, blocks / 2)))
                                  : 0.25 * (double)blocks) + 1.0 * (double)p;
      double cost = causal ? std::max((double)base * mean / at_once, len) + 0.5 * len
                           : (double)ceil_div(base * p, at_once) * len;
      if (p > 1) cost += 1.5 + (double)(heads * rows * p) * (8.0 * s.head_dim) / 4e6 / 3.6;
      if (p == 1 || cost < best) {
        best = cost;
        splits = p;
      }
    }
  }
  w.splits = (int)std::max<int64_t>(splits, 1);
  w.chunk = (int)ceil_div(blocks, w.splits);
  w.part_rows = w.splits > 1 ? w.splits * heads * rows : 0;
  return w;
}

size_t part_bytes(const rc_kv_plan* pl, int64_t part_rows) {
  // outputs, (m, l), and the number of parts (a row of the first part)
  return (size_t)part_rows * ((size_t)pl->shape.head_dim * 4 + sizeof(float2) + sizeof(int32_t));
}

// Rows that the workspace is made for: what whole sequences need for the largest
// number of queries and for smaller ones, at most half a gigabyte. A call that would
// need more takes fewer parts.
int64_t part_rows_at_most(const rc_kv_plan* pl) {
  const int64_t cap = ((int64_t)512 << 20) / (int64_t)part_bytes(pl, 1);
  int64_t most = 0, q = pl->params.max_queries;
  while (true) {
    most = std::max(most, way_of(pl, q, pl->shape.seq_blocks, false, cap).part_rows);
    if (pl->params.q_tile) most = std::max(most, way_of(pl, q, pl->params.keep_blocks, true, cap).part_rows);
    if (q == 1) return most;
    q = q > 64 ? std::max<int64_t>(q / 2, 64) : q - 1;
  }
}

rc_status_t check(const rc_kv_shape_t& s, rc_dtype_t dtype, const rc_kv_params_t* p) {
  if (!p) return RC_ERR_INVALID_ARG;
  if (s.batch < 1 || s.q_heads < 1 || s.kv_heads < 1 || s.head_dim < 1 || s.pool_blocks < 1 || s.seq_blocks < 1)
    return RC_ERR_INVALID_ARG;
  if (s.q_heads % s.kv_heads) return RC_ERR_INVALID_ARG;
  if (dtype != RC_BF16 && dtype != RC_F32) return RC_ERR_INVALID_ARG;
  if (p->max_queries < 1 || !(p->scale >= 0.0f) || !isfinite(p->scale)) return RC_ERR_INVALID_ARG;
  if (p->flags & ~RC_KV_CAUSAL) return RC_ERR_INVALID_ARG;
  if (p->q_tile != 0 && p->q_tile != 1 && p->q_tile != RC_KV_QTILE)
    return p->q_tile < 0 ? RC_ERR_INVALID_ARG : RC_ERR_UNSUPPORTED;
  if (p->q_tile == 0 ? p->keep_blocks != 0 : p->keep_blocks < 1) return RC_ERR_INVALID_ARG;
  if (p->q_tile == RC_KV_QTILE && (p->flags & RC_KV_CAUSAL) && p->keep_blocks < 3) return RC_ERR_INVALID_ARG;
  if (p->keep_blocks > 1024) return RC_ERR_UNSUPPORTED;
  if (s.head_dim != 64 && s.head_dim != 128) return RC_ERR_UNSUPPORTED;
  if (s.batch > 65535 || s.kv_heads > 32767 || s.seq_blocks > RC_KV_MAX_BLOCKS) return RC_ERR_UNSUPPORTED;
  if ((int64_t)p->max_queries * s.q_heads >= (int64_t)1 << 30) return RC_ERR_UNSUPPORTED;
  if ((int64_t)s.batch * s.seq_blocks >= (int64_t)1 << 31) return RC_ERR_UNSUPPORTED;
  return RC_OK;
}

bool at16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool at4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

rc_status_t check_cache(const rc_kv_cache_t* c) {
  if (!c || !c->k || !c->v || !c->k_scale || !c->v_scale || !c->k_mean || !c->k_mean_scale) return RC_ERR_INVALID_ARG;
  if (!at16(c->k) || !at16(c->v) || !at16(c->k_scale) || !at16(c->v_scale) || !at16(c->k_mean) ||
      !at16(c->k_mean_scale))
    return RC_ERR_ALIGNMENT;
  return RC_OK;
}

// A view of [batch][tokens][heads][dim]; strides of dimensions of size 1 do not count. The
// rows of an output must not overlap: in order of their strides, each dimension's passes
// what those before it span.
rc_status_t rows_of(const rc_kv_view_t* v, int64_t batch, int64_t tokens, int64_t heads, int64_t dim, bool out,
                    rc::KvRows* r) {
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

rc::KvGeom geometry(const rc_kv_plan* pl, const rc_kv_cache_t* c, const int32_t* table) {
  const rc_kv_shape_t& s = pl->shape;
  rc::KvGeom g;
  g.k = static_cast<uint8_t*>(c->k);
  g.v = static_cast<uint8_t*>(c->v);
  g.k_scale = c->k_scale;
  g.v_scale = c->v_scale;
  g.k_mean = c->k_mean;
  g.k_mean_scale = c->k_mean_scale;
  g.table = table;
  g.batch = s.batch;
  g.q_heads = s.q_heads;
  g.kv_heads = s.kv_heads;
  g.dim = s.head_dim;
  g.group = s.q_heads / s.kv_heads;
  g.pool_blocks = s.pool_blocks;
  g.seq_blocks = s.seq_blocks;
  return g;
}

// What rc_kv_select and rc_kv_attend check alike.
rc_status_t prepare(rc_kv_plan* pl, const rc_kv_cache_t* cache, const int32_t* table, const int32_t* kv_len,
                    int64_t max_len, int queries, const rc_kv_view_t* q, rc::KvAttendArgs* a) {
  if (!pl || !kv_len || queries < 0 || queries > pl->params.max_queries || max_len < 0) return RC_ERR_INVALID_ARG;
  if (!at4(kv_len) || (table && !at4(table))) return RC_ERR_ALIGNMENT;
  rc_status_t st = check_cache(cache);
  if (st != RC_OK) return st;
  const rc_kv_shape_t& s = pl->shape;
  st = rows_of(q, s.batch, queries, s.q_heads, s.head_dim, false, &a->q);
  if (st != RC_OK) return st;
  if (q->dtype != pl->dtype) return RC_ERR_INVALID_ARG;
  a->g = geometry(pl, cache, table);
  a->kv_len = kv_len;
  const int64_t cap = (int64_t)RC_KV_BLOCK * s.seq_blocks;
  a->max_len = (int)(max_len == 0 ? cap : std::min(max_len, cap));
  a->queries = queries;
  a->causal = (pl->params.flags & RC_KV_CAUSAL) != 0;
  a->q_tile = pl->params.q_tile;
  a->keep = pl->params.keep_blocks;
  a->tiles = a->q_tile ? (int)ceil_div(queries, a->q_tile) : 0;
  constexpr float kLog2e = 1.44269504088896340736f;
  a->scale = (pl->params.scale > 0.0f ? pl->params.scale : 1.0f / sqrtf((float)s.head_dim)) * kLog2e;
  a->lse = nullptr;
  a->blocks = nullptr;
  a->blocks_out = nullptr;
  a->splits = 1;
  a->chunk = 1;
  a->part = nullptr;
  a->part_n = nullptr;
  a->arrived = nullptr;
  a->part_ml = nullptr;
  a->out = {nullptr, 0, 0, 0};
  return RC_OK;
}

}  // namespace

extern "C" {

rc_status_t rc_kv_plan_create(rc_kv_shape_t shape, rc_dtype_t dtype, const rc_kv_params_t* params,
                              rc_kv_plan_t* out) {
  if (!out) return RC_ERR_INVALID_ARG;
  *out = nullptr;
  const rc_status_t st = check(shape, dtype, params);
  if (st != RC_OK) return st;
  rc_kv_plan* pl = new (std::nothrow) rc_kv_plan;
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

rc_status_t rc_kv_store(rc_kv_plan_t pl, hipStream_t stream, const rc_kv_cache_t* cache, const int32_t* table,
                        const int32_t* start, const int32_t* count, int tokens, const rc_kv_view_t* k,
                        const rc_kv_view_t* v) {
  if (!pl || !start || tokens < 0) return RC_ERR_INVALID_ARG;
  if (!at4(start) || (table && !at4(table)) || (count && !at4(count))) return RC_ERR_ALIGNMENT;
  rc_status_t st = check_cache(cache);
  if (st != RC_OK) return st;
  const rc_kv_shape_t& s = pl->shape;
  rc::KvStoreArgs a;
  st = rows_of(k, s.batch, tokens, s.kv_heads, s.head_dim, false, &a.k);
  if (st == RC_OK) st = rows_of(v, s.batch, tokens, s.kv_heads, s.head_dim, false, &a.v);
  if (st != RC_OK) return st;
  if (tokens == 0) return RC_OK;
  a.g = geometry(pl, cache, table);
  a.start = start;
  a.count = count;
  a.tokens = (int)std::min<int64_t>(tokens, (int64_t)RC_KV_BLOCK * s.seq_blocks);  // later ones are dropped anyway
  a.once = (int64_t)s.batch * a.tokens * s.kv_heads * s.head_dim *
               ((k->dtype == RC_BF16 ? 2 : 4) + (v->dtype == RC_BF16 ? 2 : 4)) > (int64_t)128 << 20;
  return rc::launch_kv_store(a, k->dtype == RC_BF16, v->dtype == RC_BF16, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
}

rc_status_t rc_kv_select(rc_kv_plan_t pl, hipStream_t stream, const rc_kv_cache_t* cache, const int32_t* table,
                         const int32_t* kv_len, int64_t max_len, int queries, const rc_kv_view_t* q,
                         int32_t* blocks) {
  rc::KvAttendArgs a;
  const rc_status_t st = prepare(pl, cache, table, kv_len, max_len, queries, q, &a);
  if (st != RC_OK) return st;
  if (!blocks || !a.q_tile) return RC_ERR_INVALID_ARG;
  if (!at4(blocks)) return RC_ERR_ALIGNMENT;
  if (queries == 0) return RC_OK;
  a.blocks_out = blocks;
  return rc::launch_kv_select(a, pl->dtype == RC_BF16, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
}

rc_status_t rc_kv_attend(rc_kv_plan_t pl, hipStream_t stream, const rc_kv_cache_t* cache, const int32_t* table,
                         const int32_t* kv_len, int64_t max_len, int queries, const rc_kv_view_t* q,
                         const int32_t* blocks, const rc_kv_view_t* out, float* lse) {
  rc::KvAttendArgs a;
  rc_status_t st = prepare(pl, cache, table, kv_len, max_len, queries, q, &a);
  if (st != RC_OK) return st;
  const rc_kv_shape_t& s = pl->shape;
  st = rows_of(out, s.batch, queries, s.q_heads, s.head_dim, true, &a.out);
  if (st != RC_OK) return st;
  if (out->dtype != pl->dtype || (blocks && !a.q_tile)) return RC_ERR_INVALID_ARG;
  if ((lse && !at4(lse)) || (blocks && !at4(blocks))) return RC_ERR_ALIGNMENT;
  if (queries == 0) return RC_OK;
  a.lse = lse;
  a.blocks = blocks;
  int64_t reach = ceil_div(a.max_len, RC_KV_BLOCK);
  if (blocks) reach = std::min<int64_t>(reach, a.keep);
  const Way w = way_of(pl, queries, reach, blocks != nullptr, pl->part_rows);
  a.splits = w.splits;
  a.chunk = w.chunk;
  if (w.splits > 1) {
    a.part = static_cast<float*>(pl->ws);
    a.part_ml = reinterpret_cast<float2*>(a.part + w.part_rows * s.head_dim);
    a.part_n = reinterpret_cast<int32_t*>(a.part_ml + w.part_rows);
    a.arrived = pl->arrived;
  }
  return rc::launch_kv_attend(a, w.few, pl->dtype == RC_BF16, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
}

rc_status_t rc_kv_plan_destroy(rc_kv_plan_t pl) {
  if (!pl) return RC_OK;
  hipError_t err = hipSuccess;
  if (pl->ws) err = hipFree(pl->ws);
  delete pl;
  return err == hipSuccess ? RC_OK : RC_ERR_HIP;
}

size_t rc_kv_workspace_bytes(rc_kv_plan_t pl) { return pl ? pl->ws_bytes : 0; }

}  // extern "C"
