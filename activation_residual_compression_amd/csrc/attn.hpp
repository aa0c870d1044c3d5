// Internal interface of attention over packed sequences and of the join: what the host
// code (attn_plan.cpp) hands to the kernel files attn_few / attn_many / attn_join.
#pragma once

#include "../../include/librescomp_attn.h"
#include "kv.hpp"

namespace rc {

struct AttnArgs {
  KvRows q, k, v, out;     // one batch: sb is 0
  float* lse;              // [q_tokens][q_heads] or null
  const int32_t* q_off;    // [seqs + 1]
  const int32_t* kv_off;   // [seqs + 1]
  int seqs, q_tokens, kv_tokens;
  int max_q, max_kv;       // bounds of one sequence, 1 .. tokens
  int q_heads, kv_heads, group, dim, causal;
  float scale;             // of the scores, in base 2: the plan's times log2(e)
  // Split over the keys: a group of rows that sees n keys reads them in ceil(n / chunk)
  // parts of equal length, at most `splits`, each by a block of threads of its own. With
  // one part it writes the outputs; with more, each writes partial results
  // [part][kv_heads * q_tokens * group][D] and (m, l), which are joined.
  int splits, chunk;
  // How blocks of threads find their rows: 0, from the lengths of all sequences; else every sequence has as
  // many blocks as the longest may need (the kernel for many rows: this many tiles).
  int direct;
  float* part;
  float2* part_ml;
  uint32_t* arrived;       // [groups of rows], zero between calls
  int4* joins;             // the kernel for many rows: [tiles of rows x key heads]: sequence, key head, tile, parts (0: one)
  uint16_t* halves;        // fp32, the kernel for many rows: K and V as f16, [K1, K2, V1, V2][kv_heads][kv_tokens][D],
  float* powers;           //   and their factors [kv_heads][K, V][kv_tokens]
};
// waves: 4, or more with one part; pieces: groups of 16 rows and parts of them, of a key head, at most.
hipError_t launch_attn_few(const AttnArgs& a, bool bf16, int waves, int64_t pieces, hipStream_t s);
// 128 u rows a block of threads, kg groups of waves for them; `chunk` counts tiles of 64 keys, and partial
// results are [tile and head][part][rows of a tile][D]. grid: as many blocks as there can be parts.
hipError_t launch_attn_many(const AttnArgs& a, int u, int kg, int64_t grid, hipStream_t s);
hipError_t launch_attn_many_f32(const AttnArgs& a, int64_t grid, hipStream_t s);  // the same, u = kg = 1

struct AttnJoinArgs {
  KvRows in[RC_ATTN_MAX_PARTS];
  const float* lses[RC_ATTN_MAX_PARTS];
  KvRows out;
  float* lse;              // or null
  int parts, tokens, heads, dim;
  int64_t rows;            // batch * tokens * heads
};
hipError_t launch_attn_join(const AttnJoinArgs& a, bool in_bf16, bool out_bf16, hipStream_t s);

}  // namespace rc
