// Host side of attention over packed sequences: validation, workspace, choice of the
// kernel and of the split over the keys. And of the join, which needs no plan.
#include "../../include/librescomp_attn.h"

#include <float.h>
#include <math.h>

#include <algorithm>
#include <new>

#include "attn.hpp"
#include "views.hpp"

struct rc_attn_plan {
  rc_attn_shape_t shape;
  rc_dtype_t dtype;
  rc_attn_params_t params;
  void* ws = nullptr;  // partial results: outputs, (m, l), which tile they are of; the counters; K and V as halves
  size_t ws_bytes = 0;
  int64_t part_rows = 0;        // rows of partial results that it holds
  uint32_t* arrived = nullptr;  // [kFewGroups], for the kernel for few rows
  void* halves = nullptr;       // fp32: K and V of a call as f16, and their factors
  bool many = false;            // whether the kernel for many rows can run
};

namespace {

using rc::at4;
using rc::ceil_div;
using rc::rows_of;

// Groups of rows of the kernel for few rows that may have several parts, at most.
constexpr int64_t kFewGroups = 1536;

// How a call runs: the kernel, its form, and in how many parts at most a group of rows reads
// its keys, of which length (keys; tiles of 64 keys in the kernel for many rows).
struct Way {
  bool few;
  int u, kg;
  int64_t grid;
  int splits, chunk;
  int64_t part_rows;  // rows of partial results; 0 with one part
  int direct;
};

size_t up16(size_t n) { return (n + 15) & ~(size_t)15; }

struct Call {
  int64_t seqs, q_tokens, kv_tokens, max_q, max_kv, group;
};

// The kernel for few rows: 16 rows a block of threads of u waves.
Way few_way(const rc_attn_plan* pl, const Call& c, int64_t most_rows) {
  const rc_attn_shape_t& s = pl->shape;
  const int64_t rows = c.q_tokens * s.q_heads, groups = ceil_div(c.max_q * c.group, 16), base = c.seqs * s.kv_heads * groups;
  const int64_t at_once = 512;  // blocks of threads that the CUs hold
  Way w{true, 4, 0, c.seqs * groups, 1, (int)std::max<int64_t>(c.max_kv, 1), 0, 1};
  const int64_t dense = c.q_tokens * c.group / 16 + c.seqs;  // pieces that there can be
  if (2 * dense < w.grid) {
    w.grid = dense;
    w.direct = 0;
  }
  // Few short sequences: twice as many waves and no parts (333 tokens, 24 heads of 128: 8.1 us, two parts 10.3;
  // 600 tokens, 32 heads on 8: 10.2, three parts 8.5).
  if (base <= 256 && c.max_kv <= 512) {
    w.u = 8;
    return w;
  }
  if (base > kFewGroups || rows == 0) return w;
  // equal parts of all keys that are read, one for each block of threads; each group's last part is half of one on average
  const int64_t read = c.kv_tokens * s.kv_heads * groups;
  const int64_t chunk = std::max<int64_t>(256, ceil_div(ceil_div(read, std::max(at_once - base / 2, at_once / 2)), 64) * 64);
  const int64_t most = std::min({ceil_div(c.max_kv, chunk), most_rows / rows, (int64_t)256});
  if (most <= 1) return w;
  // Parts begin at multiples of 64 keys: where the workspace limits them, rounding their length up can leave fewer.
  w.chunk = (int)std::max(chunk, ceil_div(ceil_div(c.max_kv, most), 64) * 64);
  w.splits = (int)ceil_div(c.max_kv, w.chunk);
  w.part_rows = w.splits * rows;
  // One sequence: piece w is part w % splits of group w / splits. Several are numbered without gaps.
  w.grid = groups * (c.seqs == 1 ? w.splits : std::min(c.seqs * w.splits, c.kv_tokens / w.chunk + c.seqs));
  w.direct = 0;
  return w;
}

// The kernel for many rows, in its four forms: 128 u rows a block of threads, kg groups of waves
// that share its keys. `turn` is the time in us of a turn (64 keys for each group) with 1, 2, ...
// blocks on a CU, as many as it holds; `start` a block's beginning and end; `join` the second
// launch and `move` a megabyte of partial results, written and read. Fitted to 2800 measured calls
// (180 shapes of 65 to 71000 rows, 200 to 17776 keys, 2 to 24 key heads, causal and not, each in
// every form and in 1 to 16 parts), root mean square error 6 to 8 %; the form and number of parts
// that it picks take 1.025 times as long as the best on average. For example, us: 1152 queries over
// 4608 keys, 2 x 24 heads of 128: u 2, kg 2, one part 126; u 2, kg 1 171 (146 in two parts); u 1,
// kg 1 144. 4444 over 17776, 30 heads of 64: u 2, kg 1 in 4 parts 667, in one 790. 8192 over 8192,
// 32 / 8 heads of 128: u 2, kg 1 900, kg 2 950, u 1 1087. 200 over 200, 16 x 4 / 16 heads of 128:
// u 1, kg 1 18, u 2 21.
struct Form {
  int u, kg, held;
  double turn[4], start, join, move;
};
constexpr Form kForms128[] = {{1, 1, 2, {1.46, 1.85}, 6.2, 4.4, 0.10},
                              {2, 1, 2, {2.05, 2.90}, 8.8, 3.6, 0.116},
                              {1, 2, 1, {1.90}, 6.9, 5.2, 0.10},
                              {2, 2, 1, {2.82}, 10.8, 4.3, 0.13}};
constexpr Form kForms64[] = {{1, 1, 4, {0.95, 1.27, 1.61, 1.94}, 4.2, 5.1, 0.106},
                             {2, 1, 3, {1.46, 2.02, 2.63}, 5.4, 5.5, 0.10},
                             {1, 2, 2, {1.16, 1.99}, 5.4, 5.5, 0.088},
                             {2, 2, 1, {2.01}, 6.7, 6.1, 0.108}};

// fp32, its one form, of 128 and of 64: 16 heads, 4096 keys and 256, 512 (and 768) blocks of threads.
constexpr Form kFormsF32[] = {{1, 1, 2, {3.33, 5.56}, 6.0, 8.0, 0.12}, {1, 1, 3, {2.41, 3.49, 4.68}, 5.0, 8.0, 0.12}};

double cost_of(const rc_attn_plan* pl, const Call& c, const Form& f, int64_t parts) {
  const rc_attn_shape_t& s = pl->shape;
  const bool causal = (pl->params.flags & RC_ATTN_CAUSAL) != 0;
  const double rows = 128.0 * f.u, n = (double)c.seqs;
  const double tiles = std::min(n * (double)ceil_div(c.max_q * c.group, 128 * f.u), (double)(c.q_tokens * c.group) / rows + 0.5 * n);
  const int64_t longest = ceil_div(c.max_kv, 64), chunk = ceil_div(longest, parts);
  // A tile's keys on average, in tiles of 64, and in how many parts they are read. Long sequences have more
  // tiles: half way from the average length to the longest.
  const auto length = [&](int64_t tokens, int64_t most) { return 0.5 * ((double)tokens / n + (double)std::min(most, tokens)); };
  double mean = length(c.kv_tokens, c.max_kv) / 64.0, cut = (double)parts;
  if (causal) {
    mean = std::max(mean - length(c.q_tokens, c.max_q) / 128.0, 0.5);
    cut = parts > 1 ? 1.0 + std::max(0.0, mean / (double)chunk - 0.5) : 1.0;
  }
  const double blocks = tiles * s.kv_heads * cut, turns = (double)ceil_div(chunk, f.kg), full = 256.0 * f.held;
  const auto turn = [&](double on_cu) { return f.turn[std::min(std::max((int)ceil(on_cu), 1), f.held) - 1]; };
  const auto round = [&](double blocks_at_once) { return turns * turn(blocks_at_once / 256.0) + f.start; };
  double us;
  if (blocks <= (causal ? 0.5 : 1.0) * full) {
    us = round(blocks);
  } else if (causal) {  // long ones first: the longest, or all of them and half of one at the end
    const double each = std::max(mean / cut / f.kg, 0.5) * f.turn[f.held - 1];
    us = std::max(turns * turn(std::min(blocks, full) / 256.0) + f.start, blocks / full * (each + f.start) + 0.5 * each);
  } else {  // whole rounds, and one of what is left
    const double rounds = floor(blocks / full), left = blocks - rounds * full;
    us = rounds * round(full) + (left > 0.0 ? round(left) : 0.0);
  }
  if (parts > 1) us = us * (causal ? 1.05 : 1.0) + f.join + f.move * blocks * rows * s.head_dim * 8e-6;
  return us;
}

Way many_way(const rc_attn_plan* pl, const Call& c, int64_t most_rows) {
  const rc_attn_shape_t& s = pl->shape;
  Way best{};
  double least = 0.0;
  const bool f32 = pl->dtype == RC_F32, wide = s.head_dim == 128;
  const Form* const forms = f32 ? &kFormsF32[wide ? 0 : 1] : wide ? kForms128 : kForms64;
  for (int i = 0; i < (f32 ? 1 : 4); ++i) {
    const Form& f = forms[i];
    const int64_t per = 128 * f.u;  // as many tiles of rows as there can be: a sequence ends inside of one
    const int64_t most = ceil_div(c.max_q * c.group, per), dense = std::min(c.q_tokens * c.group / per + c.seqs, c.seqs * most);
    // Among more sequences than a wave has lanes a block's rows are found by going through all of them: not where at
    // most every second block would have none (1000 sequences of 100, 32 / 8 heads of 128: 505 us,
    // by their lengths 635; 8000 of 100: 3.5 and 11.3 ms).
    const int direct = c.seqs > 64 && c.seqs * most <= 2 * dense ? (int)most : 0;
    const int64_t tiles = (direct ? c.seqs * most : dense) * s.kv_heads;
    for (const int64_t parts : {1, 2, 3, 4, 6, 8, 12, 16}) {
      if (parts > 1 && (parts * 4 > ceil_div(c.max_kv, 64) || tiles * parts * per > most_rows)) break;
      const double us = cost_of(pl, c, f, parts);
      if (least > 0.0 && us >= least) continue;
      least = us;
      best = {false, f.u, f.kg, tiles * parts, (int)parts, (int)std::max<int64_t>(ceil_div(ceil_div(c.max_kv, 64), parts), 1),
              parts > 1 ? tiles * parts * per : 0, direct};
    }
  }
  return best;
}

Way way_of(const rc_attn_plan* pl, const Call& c, int64_t most_rows) {
  const int64_t rows = c.max_q * c.group;
  // The kernel for few reads K and V once for each 16 rows, that for many has a larger tile than rows and a second
  // launch for a join. Measured in us, few and many, by what few reads: 8 heads of 128, 2000 keys, 64 rows (33 MB) 14
  // and 19, 256 rows (131 MB) 21 and 22; 24 heads, 64 rows (98 MB) 20 and 21, 128 rows (197 MB) 31 and 23; 24 heads of
  // 64, 2000 keys, 96 rows (74 MB) 15 and 18, 128 rows (98 MB) 20 and 18; 16 sequences of 500 keys, 32 rows (98 MB) 16
  // and 16, 48 rows (147 MB) 22 and 18; 64 sequences of 200 keys, 8 heads of 128, 17 rows (105 MB) 20 and 18.
  const int64_t reads = ceil_div(rows, 16) * c.kv_tokens * pl->shape.kv_heads * pl->shape.head_dim * 4;
  const bool few = rows <= 16 || reads <= (int64_t)100 << 20;
  if (pl->dtype == RC_F32) {
    // The kernel for many splits K and V before, in a launch of its own. Few and many, us: 128 rows, 2000 keys, 8 heads
    // of 64 (65 MB) 17 and 27; 256 rows (131 MB) 23 and 29; 512 rows (262 MB) 34 and 30; 256 rows, 8 heads of 128 (262
    // MB) 41 and 36; 128 rows, 200 keys, 16 x 8 heads of 64 (210 MB) 24 and 25; with half of a tile or less 64 rows,
    // 2000 keys, 16 x 8 heads of 128 (1 GB) 153 and 163.
    return rows <= 64 || 2 * reads <= (int64_t)200 << 20 || !pl->many ? few_way(pl, c, most_rows) : many_way(pl, c, most_rows);
  }
  return few ? few_way(pl, c, most_rows) : many_way(pl, c, most_rows);
}

// Bytes of K and V of `keys` tokens as two f16 each, and of their factors.
size_t half_bytes(const rc_attn_plan* pl, int64_t keys) {
  return (size_t)keys * pl->shape.kv_heads * ((size_t)pl->shape.head_dim * 8 + 8);
}
// The kernel for many rows of fp32 is there for plans whose K and V as halves take no more than this.
constexpr size_t kMostHalves = (size_t)4 << 30;

// Bytes of partial results: outputs, (m, l), and for each 128 rows or more which tile they are.
size_t part_bytes(const rc_attn_plan* pl, int64_t part_rows) {
  return (size_t)part_rows * ((size_t)pl->shape.head_dim * 4 + sizeof(float2)) + (size_t)ceil_div(part_rows, 128) * sizeof(int4);
}

// Rows of partial results that the workspace is made for: what calls of one sequence, of
// all, and of powers of two between need, with few and with all queries, at most half a
// gigabyte. A call that would need more takes fewer parts.
int64_t part_rows_at_most(const rc_attn_plan* pl) {
  const rc_attn_shape_t& s = pl->shape;
  const int64_t cap = ((int64_t)512 << 20) / ((int64_t)s.head_dim * 4 + 9), group = s.q_heads / s.kv_heads;
  int64_t most = 0;
  for (int64_t n = 1;; n = std::min<int64_t>(2 * n, s.max_seqs)) {
    for (int64_t q = 1;; q = std::min<int64_t>(2 * q, s.max_queries)) {
      if (q >= n) most = std::max(most, way_of(pl, {n, q, s.max_keys, ceil_div(q, n), s.max_keys, group}, cap).part_rows);
      if (q == s.max_queries) break;
    }
    if (n == s.max_seqs) return most;
  }
}

// Threads of the call's largest launch: of the kernel, of the join of its parts, of the split of K and V before it.
int64_t most_threads(const rc_attn_plan* pl, const Call& c, const Way& w) {
  const rc_attn_shape_t& s = pl->shape;
  if (w.few) return w.grid * s.kv_heads * 64 * w.u;
  const int64_t join = w.splits > 1 ? w.grid / w.splits * (w.u * s.head_dim / 32) * 256 : 0;
  const int64_t halves = pl->dtype == RC_F32 ? (c.kv_tokens * s.kv_heads * (s.head_dim / 8) + 255) / 256 * 256 : 0;
  return std::max({w.grid * 256 * w.kg, join, halves});
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
  const size_t halves = half_bytes(pl, shape.max_keys);
  pl->many = dtype == RC_BF16 || halves <= kMostHalves;
  pl->part_rows = part_rows_at_most(pl);
  const size_t parts = pl->part_rows ? part_bytes(pl, pl->part_rows) : 0, counts = parts ? kFewGroups * sizeof(uint32_t) : 0;
  const bool halved = dtype == RC_F32 && pl->many && (int64_t)shape.max_queries * (shape.q_heads / shape.kv_heads) > 64;
  pl->ws_bytes = up16(parts + counts) + (halved ? halves : 0);
  if (pl->ws_bytes) {
    if (!rc::allocate(&pl->ws, pl->ws_bytes)) {
      delete pl;
      return RC_ERR_HIP;
    }
    if (halved) pl->halves = static_cast<char*>(pl->ws) + up16(parts + counts);
  }
  if (counts) {
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
  const Call c{seqs, q_tokens, kv_tokens, a.max_q, a.max_kv, a.group};
  const Way w = way_of(pl, c, pl->part_rows);
  if (most_threads(pl, c, w) >= (int64_t)1 << 32) return RC_ERR_UNSUPPORTED;  // a launch would run fewer, without an error
  a.splits = w.splits;
  a.direct = w.direct;
  a.chunk = w.chunk;
  a.part = static_cast<float*>(pl->ws);
  a.part_ml = reinterpret_cast<float2*>(a.part + w.part_rows * s.head_dim);
  a.joins = reinterpret_cast<int4*>(a.part_ml + w.part_rows);
  a.arrived = pl->arrived;
  if (!w.few && pl->dtype == RC_F32) {
    a.halves = static_cast<uint16_t*>(pl->halves);
    a.powers = reinterpret_cast<float*>(a.halves + (int64_t)4 * s.kv_heads * kv_tokens * s.head_dim);
    return rc::launch_attn_many_f32(a, w.grid, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
  }
  if (!w.few) return rc::launch_attn_many(a, w.u, w.kg, w.grid, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
  return rc::launch_attn_few(a, pl->dtype == RC_BF16, w.u, w.grid, stream) == hipSuccess ? RC_OK : RC_ERR_HIP;
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
  const __int128 rows = (__int128)((int64_t)batch * tokens) * heads;  // up to 2^93
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
  a.rows = (int64_t)rows;
  return rc::launch_attn_join(a, outs[0].dtype == RC_BF16, out->dtype == RC_BF16, stream) == hipSuccess ? RC_OK
                                                                                                       : RC_ERR_HIP;
}

}  // extern "C"
