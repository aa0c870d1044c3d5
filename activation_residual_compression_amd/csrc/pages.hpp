// Internal interface of the cache's pages: what the host code (pages_plan.cpp) hands to
// the kernels (pages.hip).
#pragma once

#include "../../include/librescomp_pages.h"
#include "kv.hpp"

namespace rc {

// The parts of a cache, each [pool_blocks][bytes of a block], and those bytes.
constexpr int kPageParts = 6;
struct PageParts {
  char* at[kPageParts];  // k, v, k_mean, k_scale, v_scale, k_mean_scale
};
struct PageGeom {
  int slots, pool_blocks, seq_blocks;
  int bytes[kPageParts];  // the first three multiples of 64, the others of 4
};

// Device workspace of a plan. writers, first: for reserve, 0 and INT32_MAX between calls.
struct PageWork {
  int32_t* writers;  // [pool]: entries of the call that would write a shared block
  int32_t* first;    // [pool]: the first of them
  int32_t* list;     // [pool]: free blocks given out; compact: sources, from the end destinations
  int32_t* old;      // [pool]: what those replace, or -1
  int32_t* place;    // [pool]: compact: where a block goes
  int2* pairs;       // [slots]: reserve: contents to copy (from, to), from < 0: none
  int32_t* count;    // [1]: compact: blocks that move
  int32_t* rows;     // [slots][seq_blocks]: fork: the new rows
};

hipError_t launch_pages_reserve(const PageGeom& g, const PageWork& w, const PageParts& cache, int32_t* refs,
                                int32_t* table, const int32_t* start, const int32_t* tokens, int32_t* missing,
                                hipStream_t s);
hipError_t launch_pages_fork(const PageGeom& g, const PageWork& w, int32_t* refs, int32_t* table, const int32_t* source,
                             const int32_t* length, hipStream_t s);
hipError_t launch_pages_free(const PageGeom& g, int32_t* refs, int32_t* table, const int32_t* keep, hipStream_t s);
hipError_t launch_pages_compact(const PageGeom& g, const PageWork& w, const PageParts& cache, int32_t* refs,
                                int32_t* table, int32_t* used, int32_t* moved, hipStream_t s);
hipError_t launch_pages_copy(const PageGeom& g, const PageParts& from, const PageParts& to, const int32_t* src,
                             const int32_t* dst, int count, hipStream_t s);

}  // namespace rc
