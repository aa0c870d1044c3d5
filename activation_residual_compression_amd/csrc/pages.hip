// Pages of the key/value cache: reserving, forking, freeing, compacting, copying.
//
// The decisions (which block goes where) are made by one block of threads in a fixed order,
// by prefix sums, so they are the same every time; the contents are moved by as many blocks
// of threads as there is data. Counts of holders change by atomic additions of whole
// numbers, whose order does not matter.
#include <hip/hip_runtime.h>

#include "device_common.hpp"
#include "pages.hpp"

namespace rc {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;

__device__ __forceinline__ int blocks_of(int64_t tokens) { return (int)((tokens + RC_KV_BLOCK - 1) / RC_KV_BLOCK); }

// Reads past the CU's own cache: what this call's atomics have left there.
__device__ __forceinline__ int fresh(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Sum of x over the threads before this one, and over all; called by the whole block of threads.
__device__ __forceinline__ int before(int x, int* wave_sums, int& all) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int sum = x;
#pragma unroll
  for (int d = 1; d < 64; d *= 2) {
    const int y = __shfl_up(sum, d);
    if (lane >= d) sum += y;
  }
  __syncthreads();  // the last call's sums are read
  if (lane == 63) wave_sums[wave] = sum;
  __syncthreads();
  int base = 0;
  all = 0;
#pragma unroll
  for (int w = 0; w < kWaves; ++w) {
    if (w < wave) base += wave_sums[w];
    all += wave_sums[w];
  }
  return base + sum - x;
}

// ------------------------------------------------------------------ contents
// Bytes of a part that a block of threads copies: 16 KB.
constexpr int kChunk = 16384;
// Chunks of the two large parts; the others go with chunk 0.
__host__ __device__ __forceinline__ int chunks_of(const PageGeom& g) {
  return (g.bytes[0] + kChunk - 1) / kChunk + (g.bytes[1] + kChunk - 1) / kChunk;
}
// Copies chunk `chunk` of block src to block dst; 256 threads. The stores go past the caches, which the data
// would fill and nobody read (500 blocks of 24 heads of 128, 397 MB read and written, the source in the last-level
// cache: 58 us, 6.9 TB/s, stores through it 82; all from HBM: 80, 83). Loads past it too are faster from HBM (76) and
// slower from the cache (76).
__device__ __forceinline__ void copy_chunk(const PageGeom& g, const PageParts& from, const PageParts& to, int src, int dst,
                                           int chunk) {
  const int of_k = (g.bytes[0] + kChunk - 1) / kChunk, part = chunk >= of_k, at = (chunk - part * of_k) * kChunk;
  const int n = min(kChunk, g.bytes[part] - at);
  const u32x4* a = reinterpret_cast<const u32x4*>(from.at[part] + (int64_t)src * g.bytes[part] + at);
  u32x4* b = reinterpret_cast<u32x4*>(to.at[part] + (int64_t)dst * g.bytes[part] + at);
  u32x4 x[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((int)(threadIdx.x + 256 * i) * 16 < n) x[i] = a[threadIdx.x + 256 * i];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    if ((int)(threadIdx.x + 256 * i) * 16 < n) __builtin_nontemporal_store(x[i], &b[threadIdx.x + 256 * i]);
  if (chunk) return;
#pragma unroll
  for (int p = 2; p < kPageParts; ++p) {
    const uint32_t* c = reinterpret_cast<const uint32_t*>(from.at[p] + (int64_t)src * g.bytes[p]);
    uint32_t* d = reinterpret_cast<uint32_t*>(to.at[p] + (int64_t)dst * g.bytes[p]);
    for (int i = threadIdx.x; i < g.bytes[p] / 4; i += 256) d[i] = c[i];
  }
}

__global__ __launch_bounds__(256) void pages_copy_kernel(PageGeom g, PageParts from, PageParts to, const int32_t* src,
                                                         const int32_t* dst, int chunks, int pair0, int chunk0) {
  // Blocks of threads go to the 8 XCDs in turn; each gets a run of the work (77 us, in turn 80).
  const int runs = gridDim.x / 8, w = (int)blockIdx.x < 8 * runs ? (int)blockIdx.x % 8 * runs + (int)blockIdx.x / 8 : (int)blockIdx.x;
  const int i = pair0 + (chunk0 + w) / chunks, chunk = (chunk0 + w) % chunks;
  const int p = src[i], q = dst[i];
  if ((unsigned)p >= (unsigned)g.pool_blocks || (unsigned)q >= (unsigned)g.pool_blocks) return;
  copy_chunk(g, from, to, p, q, chunk);
}

// ------------------------------------------------------------------ reserve
// The entries that a call touches, in order: those of slot 0, of slot 1, ... Taken 1024 slots
// and 1024 entries at a time.
struct Entries {
  const PageGeom& g;
  const int32_t* start;
  const int32_t* tokens;
  int* sums;       // [kWaves]
  int* ends;       // [kThreads]: entries up to and with the slot's
  int* firsts;     // [kThreads]: its first entry

  // Takes the slots from s0 on; returns their entries' number.
  __device__ __forceinline__ int take(int s0) const {
    const int s = s0 + threadIdx.x;
    int j0 = 0, n = 0;
    if (s < g.slots) {
      const int at = start[s], more = tokens[s];
      if (at >= 0 && more > 0) {
        j0 = min(at / RC_KV_BLOCK, g.seq_blocks);
        n = max(min(blocks_of((int64_t)at + more), g.seq_blocks) - j0, 0);
      }
    }
    int all;
    const int lead = before(n, sums, all);
    ends[threadIdx.x] = lead + n;
    firsts[threadIdx.x] = j0;
    __syncthreads();
    return all;
  }
  // Slot (from s0 on) and place in its row of entry e of `all`.
  __device__ __forceinline__ void find(int e, int all, int& slot, int& j) const {
    int lo = 0;  // the first slot whose entries end after e
#pragma unroll
    for (int step = kThreads / 2; step; step /= 2)
      if (e < all && ends[lo + step - 1] <= e) lo += step;
    slot = lo;
    j = e < all ? firsts[lo] + e - (lo ? ends[lo - 1] : 0) : 0;
  }
  // Calls what(live, slot, j) for every entry, by all threads together.
  template <typename F>
  __device__ __forceinline__ void each(F&& what) const {
    for (int s0 = 0; s0 < g.slots; s0 += kThreads) {
      const int all = take(s0);
      for (int e0 = 0; e0 < all; e0 += kThreads) {
        int s, j;
        find(e0 + threadIdx.x, all, s, j);
        what(e0 + (int)threadIdx.x < all, s0 + s, j);
      }
      __syncthreads();
    }
  }
};

__global__ __launch_bounds__(kThreads) void pages_reserve_kernel(PageGeom g, PageWork w, int32_t* refs, int32_t* table,
                                                                 const int32_t* start, const int32_t* tokens,
                                                                 int32_t* missing) {
  __shared__ int sums[kWaves], ends[kThreads], firsts[kThreads];
  const Entries entries{g, start, tokens, sums, ends, firsts};
  // The entry's block, -1 without one; refs and (but for the entry itself) the table stay as
  // they are until all is decided.
  const auto block_at = [&](bool live, int s, int j) {
    const int p = live ? table[(int64_t)s * g.seq_blocks + j] : -1;
    return (unsigned)p < (unsigned)g.pool_blocks ? p : -1;
  };
  // The free ones among four blocks of each thread from block p0 on; returns how many all threads have, and
  // gives those before the need-th to `to`.
  const auto find_free = [&](const int (&count)[4], int p0, int found, int need, int* to) {
    const int p = p0 + 4 * threadIdx.x;
    int n = 0, all;
#pragma unroll
    for (int i = 0; i < 4; ++i) n += p + i < g.pool_blocks && count[i] <= 0;
    int at = found + before(n, sums, all);
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (p + i < g.pool_blocks && count[i] <= 0) {
        if (at < need) to[at] = p + i;
        ++at;
      }
    return all;
  };
  const auto counts = [&](int p0, int (&count)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) count[i] = refs[min(p0 + (int)(4 * threadIdx.x) + i, g.pool_blocks - 1)];
  };
  for (int s = threadIdx.x; s < g.slots; s += kThreads) w.pairs[s] = make_int2(-1, -1);
  if (g.slots <= kThreads) {
    // A thread for each entry, if there are as many: what it has read stays in its registers (64 sequences,
    // five tokens each: 5.1 us, by the passes below 12.7).
    int count[4];
    counts(0, count);  // in flight meanwhile
    const int all = entries.take(0);
    if (all <= kThreads) {
      __shared__ int list[kThreads];
      int s, j;
      const bool live = (int)threadIdx.x < all;
      entries.find(threadIdx.x, all, s, j);
      const int p = block_at(live, s, j), holders = p >= 0 ? refs[p] : 0;
      const bool shared = holders > 1;
      bool keeps = false;
      if (__syncthreads_or(shared)) {  // who would write each shared block, in LDS by the block's number
        constexpr int SLOTS = 2 * kThreads;
        __shared__ int block[SLOTS], writers[SLOTS], first[SLOTS];
        for (int i = threadIdx.x; i < SLOTS; i += kThreads) {
          block[i] = -1;
          writers[i] = 0;
          first[i] = INT32_MAX;
        }
        __syncthreads();
        uint32_t at = 0;
        if (shared) {
          at = ((uint32_t)p * 2654435761u) >> 21;  // of SLOTS
          for (;; at = (at + 1) % SLOTS) {  // ends: at most half of the slots are taken
            const int was = atomicCAS(&block[at], -1, p);
            if (was == -1 || was == p) break;
          }
          atomicAdd(&writers[at], 1);
          atomicMin(&first[at], s * g.seq_blocks + j);
        }
        __syncthreads();
        keeps = shared && writers[at] == holders && first[at] == s * g.seq_blocks + j;
      }
      const bool mine = live && (p < 0 || (shared && !keeps));
      int need;
      const int rank = before(mine, sums, need);
      int found = 0;
      for (int p0 = 0; p0 < g.pool_blocks && found < need; p0 += 4 * kThreads) {
        if (p0) counts(p0, count);
        found += find_free(count, p0, found, need, list);
      }
      if (missing && threadIdx.x == 0) *missing = max(need - found, 0);
      __syncthreads();
      if (found >= need && mine) {
        const int q = list[rank];
        if (p >= 0 && (int64_t)j * RC_KV_BLOCK < start[s]) w.pairs[s] = make_int2(p, q);
        table[(int64_t)s * g.seq_blocks + j] = q;
        refs[q] = 1;
        if (p >= 0) atomicSub(&refs[p], 1);
      }
      return;
    }
    __syncthreads();
  }
  // who would write each shared block
  entries.each([&](bool live, int s, int j) {
    const int p = block_at(live, s, j);
    if (p >= 0 && refs[p] > 1) {
      atomicAdd(&w.writers[p], 1);
      atomicMin(&w.first[p], s * g.seq_blocks + j);
    }
  });
  __threadfence();
  __syncthreads();
  // An entry needs a block if it has none, or a shared one that it does not keep.
  const auto needs = [&](bool live, int p, int s, int j) {
    if (!live || p < 0) return live;
    const int holders = refs[p];
    return holders > 1 && !(fresh(&w.writers[p]) == holders && fresh(&w.first[p]) == s * g.seq_blocks + j);
  };
  int need = 0;
  entries.each([&](bool live, int s, int j) {
    int all;
    before(needs(live, block_at(live, s, j), s, j), sums, all);
    need += all;
  });
  // the first `need` free blocks
  int found = 0;
  for (int p0 = 0; p0 < g.pool_blocks && found < need; p0 += 4 * kThreads) {
    int count[4];
    counts(p0, count);
    found += find_free(count, p0, found, need, w.list);
  }
  const bool enough = found >= need;
  if (missing && threadIdx.x == 0) *missing = enough ? 0 : need - found;
  __syncthreads();
  if (!enough) {
    entries.each([&](bool live, int s, int j) {
      const int p = block_at(live, s, j);
      if (p >= 0 && refs[p] > 1) {
        w.writers[p] = 0;
        w.first[p] = INT32_MAX;
      }
    });
    return;
  }
  int rank = 0;
  entries.each([&](bool live, int s, int j) {
    int all;
    const int p = block_at(live, s, j);
    const bool mine = needs(live, p, s, j);
    const int at = rank + before(mine, sums, all);
    rank += all;
    if (mine) {
      const int q = w.list[at];
      w.old[at] = p;
      if (p >= 0 && (int64_t)j * RC_KV_BLOCK < start[s]) w.pairs[s] = make_int2(p, q);
      table[(int64_t)s * g.seq_blocks + j] = q;
    }
  });
  __syncthreads();
  for (int k = threadIdx.x; k < need; k += kThreads) {
    refs[w.list[k]] = 1;
    const int p = w.old[k];
    if (p >= 0) {  // every shared block that the call counted is given up by one entry at least
      atomicSub(&refs[p], 1);
      w.writers[p] = 0;
      w.first[p] = INT32_MAX;
    }
  }
}

__global__ __launch_bounds__(256) void pages_pairs_kernel(PageGeom g, PageParts cache, const int2* pairs, int chunks, int64_t first) {
  const uint32_t at = (uint32_t)first + blockIdx.x;  // slots * chunks: under 2^31
  const int2 pair = pairs[at / chunks];
  if (pair.x >= 0) copy_chunk(g, cache, cache, pair.x, pair.y, at % chunks);
}

// ------------------------------------------------------------------ fork, free
// The new rows, and what becomes of the counts.
__global__ __launch_bounds__(256) void pages_fork_kernel(PageGeom g, int32_t* rows, int32_t* refs, const int32_t* table,
                                                         const int32_t* source, const int32_t* length) {
  const int s = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x, from = source[s];
  if ((unsigned)from >= (unsigned)g.slots || j >= g.seq_blocks) return;
  const int was = table[(int64_t)s * g.seq_blocks + j];
  const int now = j < blocks_of(max(length[s], 0)) ? table[(int64_t)from * g.seq_blocks + j] : -1;
  if (was != now) {
    if ((unsigned)was < (unsigned)g.pool_blocks) atomicSub(&refs[was], 1);
    if ((unsigned)now < (unsigned)g.pool_blocks) atomicAdd(&refs[now], 1);
  }
  rows[(int64_t)s * g.seq_blocks + j] = now;
}
__global__ __launch_bounds__(256) void pages_rows_kernel(PageGeom g, const int32_t* rows, int32_t* table,
                                                         const int32_t* source) {
  const int s = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  if ((unsigned)source[s] >= (unsigned)g.slots || j >= g.seq_blocks) return;
  table[(int64_t)s * g.seq_blocks + j] = rows[(int64_t)s * g.seq_blocks + j];
}

// Both at once, by one block of threads, for tables of up to kForkEntries entries (2304 entries:
// 4.0 us, by the two above 4.8 and a launch).
constexpr int kForkEach = 8, kForkEntries = kForkEach * kThreads;
__global__ __launch_bounds__(kThreads) void pages_fork_small_kernel(PageGeom g, int32_t* refs, int32_t* table,
                                                                    const int32_t* source, const int32_t* length) {
  int now[kForkEach], was[kForkEach];
#pragma unroll
  for (int k = 0; k < kForkEach; ++k) {
    const int i = threadIdx.x + k * kThreads, s = i / g.seq_blocks, j = i % g.seq_blocks;
    const int from = s < g.slots ? source[s] : -1;
    was[k] = now[k] = -1;
    if ((unsigned)from < (unsigned)g.slots) {
      was[k] = table[i];
      if (j < blocks_of(max(length[s], 0))) now[k] = table[(int64_t)from * g.seq_blocks + j];
    }
  }
  __syncthreads();  // all rows are read
#pragma unroll
  for (int k = 0; k < kForkEach; ++k) {
    if (was[k] == now[k]) continue;
    if ((unsigned)was[k] < (unsigned)g.pool_blocks) atomicSub(&refs[was[k]], 1);
    if ((unsigned)now[k] < (unsigned)g.pool_blocks) atomicAdd(&refs[now[k]], 1);
    table[threadIdx.x + k * kThreads] = now[k];
  }
}

__global__ __launch_bounds__(256) void pages_free_kernel(PageGeom g, int32_t* refs, int32_t* table, const int32_t* keep) {
  const int s = blockIdx.y, j = blockIdx.x * 256 + threadIdx.x;
  if (j >= g.seq_blocks || j < blocks_of(max(keep[s], 0))) return;
  const int p = table[(int64_t)s * g.seq_blocks + j];
  if ((unsigned)p < (unsigned)g.pool_blocks) atomicSub(&refs[p], 1);
  if (p != -1) table[(int64_t)s * g.seq_blocks + j] = -1;
}

// ------------------------------------------------------------------ compact
// Two launches, the places and the moves. 1024 blocks of 8 heads of 128 in use in a pool of 2048, half of them
// to be moved: 4.8 and 23.6 us (5.7 TB/s).
__global__ __launch_bounds__(kThreads) void pages_place_kernel(PageGeom g, PageWork w, const int32_t* refs, int32_t* used,
                                                               int32_t* moved) {
  __shared__ int sums[kWaves];
  int n = 0, count;
  for (int p = threadIdx.x; p < g.pool_blocks; p += kThreads) n += refs[p] > 0;
  before(n, sums, count);
  int above = 0, holes = 0;  // so far
  for (int p0 = 0; p0 < g.pool_blocks; p0 += kThreads) {
    const int p = p0 + threadIdx.x;
    const bool in = p < g.pool_blocks, use = in && refs[p] > 0;
    int all;
    // one of the two at most: before `count` only holes are counted, from there on only blocks in use
    const int lead = before(in && (p < count ? !use : use), sums, all);
    // the step that holds `count` has both: its holes come first
    const int split = min(max(count - p0, 0), kThreads);
    int holes_here = all;
    if (split < kThreads) {
      __shared__ int at_split;
      __syncthreads();
      if (threadIdx.x == split) at_split = lead;
      __syncthreads();
      holes_here = at_split;
    }
    if (in) {
      if (p < count && !use) w.list[g.pool_blocks - 1 - (holes + lead)] = p;
      if (p >= count && use) w.list[above + lead - holes_here] = p;
      const int to = use ? p : -1;
      w.place[p] = to;
      if (moved) moved[p] = to;
    }
    holes += holes_here;
    above += all - holes_here;
  }
  __syncthreads();
  for (int k = threadIdx.x; k < above; k += kThreads) {
    const int p = w.list[k], to = w.list[g.pool_blocks - 1 - k];
    w.place[p] = to;
    if (moved) moved[p] = to;
  }
  if (threadIdx.x == 0) {
    *w.count = above;
    if (used) *used = count;
  }
}

__global__ __launch_bounds__(256) void pages_move_kernel(PageGeom g, PageWork w, PageParts cache, int32_t* refs,
                                                         int32_t* table, int table_blocks, int chunks) {
  if ((int)blockIdx.x < table_blocks) {
    const int64_t all = (int64_t)g.slots * g.seq_blocks;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < all; i += (int64_t)table_blocks * 256) {
      const int p = table[i];
      if ((unsigned)p < (unsigned)g.pool_blocks) {
        const int to = w.place[p];
        if (to >= 0 && to != p) table[i] = to;
      }
    }
    return;
  }
  const int64_t work = (int64_t)*w.count * chunks;
  for (int64_t i = blockIdx.x - table_blocks; i < work; i += gridDim.x - table_blocks) {
    const int k = (int)(i / chunks), chunk = (int)(i % chunks);
    const int src = w.list[k], dst = w.list[g.pool_blocks - 1 - k];
    copy_chunk(g, cache, cache, src, dst, chunk);
    if (chunk == 0 && threadIdx.x == 0) {
      refs[dst] = refs[src];
      refs[src] = 0;
    }
  }
}

dim3 row_grid(const PageGeom& g) { return dim3((unsigned)((g.seq_blocks + 255) / 256), (unsigned)g.slots); }

}  // namespace

hipError_t launch_pages_reserve(const PageGeom& g, const PageWork& w, const PageParts& cache, int32_t* refs,
                                int32_t* table, const int32_t* start, const int32_t* tokens, int32_t* missing,
                                hipStream_t s) {
  pages_reserve_kernel<<<1, kThreads, 0, s>>>(g, w, refs, table, start, tokens, missing);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int chunks = chunks_of(g);
  return launch_all((int64_t)g.slots * chunks, [&](int64_t first, unsigned blocks) {
    pages_pairs_kernel<<<blocks, 256, 0, s>>>(g, cache, w.pairs, chunks, first);
  });
}

hipError_t launch_pages_fork(const PageGeom& g, const PageWork& w, int32_t* refs, int32_t* table, const int32_t* source,
                             const int32_t* length, hipStream_t s) {
  if ((int64_t)g.slots * g.seq_blocks <= kForkEntries) {
    pages_fork_small_kernel<<<1, kThreads, 0, s>>>(g, refs, table, source, length);
    return hipGetLastError();
  }
  pages_fork_kernel<<<row_grid(g), 256, 0, s>>>(g, w.rows, refs, table, source, length);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  pages_rows_kernel<<<row_grid(g), 256, 0, s>>>(g, w.rows, table, source);
  return hipGetLastError();
}

hipError_t launch_pages_free(const PageGeom& g, int32_t* refs, int32_t* table, const int32_t* keep, hipStream_t s) {
  pages_free_kernel<<<row_grid(g), 256, 0, s>>>(g, refs, table, keep);
  return hipGetLastError();
}

hipError_t launch_pages_compact(const PageGeom& g, const PageWork& w, const PageParts& cache, int32_t* refs,
                                int32_t* table, int32_t* used, int32_t* moved, hipStream_t s) {
  pages_place_kernel<<<1, kThreads, 0, s>>>(g, w, refs, used, moved);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  const int64_t entries = (int64_t)g.slots * g.seq_blocks;
  const int table_blocks = (int)((entries + 255) / 256 < 256 ? (entries + 255) / 256 : 256);
  const int chunks = chunks_of(g);
  const int64_t most = (int64_t)(g.pool_blocks / 2) * chunks;
  const int movers = (int)(most < 1 ? 1 : most < 4096 ? most : 4096);
  pages_move_kernel<<<(unsigned)(table_blocks + movers), 256, 0, s>>>(g, w, cache, refs, table, table_blocks, chunks);
  return hipGetLastError();
}

hipError_t launch_pages_copy(const PageGeom& g, const PageParts& from, const PageParts& to, const int32_t* src,
                             const int32_t* dst, int count, hipStream_t s) {
  const int chunks = chunks_of(g);
  return launch_all((int64_t)count * chunks, [&](int64_t first, unsigned blocks) {
    pages_copy_kernel<<<blocks, 256, 0, s>>>(g, from, to, src, dst, chunks, (int)(first / chunks), (int)(first % chunks));
  });
}

}  // namespace rc
