// Internal interface of the 8-bit key/value cache: what the host code
// (kv_plan.cpp) hands to the kernel files kv_store / kv_select / kv_attend.
#pragma once

#include <hip/hip_runtime_api.h>
#include <stdint.h>

#include "../../include/librescomp_kv.h"

namespace rc {

constexpr int kKvBlock = RC_KV_BLOCK;
constexpr int kKvQTile = RC_KV_QTILE;
constexpr int kKvEMin = -40, kKvEMax = 44;  // exponents of a block's scale

// Rows [batch][tokens][heads][D]; strides in elements.
struct KvRows {
  void* data;
  int64_t sb, st, sh;
};

// What every kernel of the cache needs to find a block.
struct KvGeom {
  uint8_t* k;
  uint8_t* v;
  float* k_scale;
  float* v_scale;
  int8_t* k_mean;
  float* k_mean_scale;
  const int32_t* table;  // [batch][seq_blocks] or null
  int batch, q_heads, kv_heads, dim, group;
  int pool_blocks, seq_blocks;
};

struct KvStoreArgs {
  KvGeom g;
  KvRows k, v;
  const int32_t* start;
  const int32_t* count;  // or null
  int tokens;
  bool once;  // the inputs are larger than half the last-level cache (256 MB)
};
hipError_t launch_kv_store(const KvStoreArgs& a, bool k_bf16, bool v_bf16, hipStream_t s);

struct KvAttendArgs {
  KvGeom g;
  KvRows q, out;
  float* lse;             // or null
  const int32_t* kv_len;
  const int32_t* blocks;  // [batch][kv_heads][tiles][keep] or null
  int32_t* blocks_out;    // rc_kv_select
  int max_len;            // bound of kv_len, at most 64 * seq_blocks
  int queries, causal;
  int q_tile, keep, tiles;
  float scale;            // of the scores, in base 2: the plan's times log2(e)
  // Split over the keys: a group of rows that reads n blocks does so in
  // ceil(n / chunk) parts of equal length, at most `splits`, each by a block of
  // threads of its own. With one part it writes the outputs; with more, each writes
  // partial results [part][batch * kv_heads * rows][D] and (m, l), which are joined.
  int splits, chunk;
  float* part;
  float2* part_ml;
  int32_t* part_n;   // kernel for many rows: parts of each row, for the launch that joins them
  uint32_t* arrived; // kernel for few rows: parts done of each group, 0 between calls; the last one joins them
};
hipError_t launch_kv_select(const KvAttendArgs& a, bool bf16, hipStream_t s);
// few: the kernel for few rows (16 rows of a key head per block), else the one
// for many (64 rows, or 32 in fp32 at 128 channels).
hipError_t launch_kv_attend(const KvAttendArgs& a, bool few, bool bf16, hipStream_t s);

}  // namespace rc
