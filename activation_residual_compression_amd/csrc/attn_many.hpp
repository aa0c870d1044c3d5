// Device helpers of the two kernels of attention over packed sequences for many rows, and the join
// of their partial results.
#pragma once

#include "attn_device.hpp"

namespace rc {
namespace {

typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr int kTile = 64;       // keys, as parts of the keys are counted
constexpr int kMostParts = 16;  // of a tile of rows

// A tile in LDS: rows of 2 D bytes without gaps, as the loads that write them lay them. The
// 16-byte chunks of a row are in the order c ^ turn(row), so that what a read takes in one cycle,
// a column of 16 chunks (K) or four rows of 64 bytes (V), meets different banks.
template <int D>
__device__ __forceinline__ int k_turn(int row) { return D == 128 ? row & 15 : row >> 1 & 7; }
template <int D>
__device__ __forceinline__ int v_turn(int row) { return D == 128 ? (row & 3) << 2 : (row >> 1 & 1) << 2; }

// 16 bytes a lane from memory into LDS at `to` (one for the wave) + 16 lane, past the
// registers, from base + offset or from an address of each lane. The compiler's own form of this
// makes every later read of LDS wait for it; here the wait is the caller's (vmcnt), once a tile.
// Nothing else in these kernels uses m0.
__device__ __forceinline__ void load_lds(uint32_t to, uint32_t offset, const void* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory", "m0");
}
__device__ __forceinline__ void load_lds(uint32_t to, const void* at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(at) : "memory", "m0");
}

__device__ __forceinline__ void load_lds_4(uint32_t to, const void* at) {  // 4 bytes a lane
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dword %1, off" ::"s"(to), "v"(at) : "memory", "m0");
}

// vmcnt(0). In the form that the compiler understands: it would else go on waiting, tile after
// tile, for loads from before the loop, and with them for the ones of load_lds.
__device__ __forceinline__ void wait_loads() {
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt(0x0F70);
  asm volatile("" ::: "memory");
}

// The thread's number, as if not known yet: what is worked out from it anew, where it is needed,
// takes no registers through the loops.
__device__ __forceinline__ int thread_again() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

// The sum of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float sum_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

// Sum of x over the wave's lanes, the same in all: inside rows of 16 lanes by moves between
// neighbours, over the rows by scalars.
__device__ __forceinline__ int wave_total(int x) {
  x += (int)dpp_u32<kQuadXor1>((uint32_t)x);
  x += (int)dpp_u32<kQuadXor2>((uint32_t)x);
  x += (int)dpp_u32<kHalfMirror>((uint32_t)x);
  x += (int)dpp_u32<kRowMirror>((uint32_t)x);
  return __builtin_amdgcn_readlane(x, 0) + __builtin_amdgcn_readlane(x, 16) + __builtin_amdgcn_readlane(x, 32) + __builtin_amdgcn_readlane(x, 48);
}
__device__ __forceinline__ int wave_top(int x) {  // the largest, of numbers that are not negative
  x = (int)group_max_u32<16>((uint32_t)x);
  return max(max(__builtin_amdgcn_readlane(x, 0), __builtin_amdgcn_readlane(x, 16)),
             max(__builtin_amdgcn_readlane(x, 32), __builtin_amdgcn_readlane(x, 48)));
}

// Which rows a block of threads does; called by a whole wave. Tiles of rows are given out by
// their number in their sequence, highest first over all sequences: with a causal mask the long
// ones first, and without it those of the long sequences.
struct Place {
  int b, h, tile;  // b < 0: none
};
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int queries, int rows_per) {
  return (queries * a.group + rows_per - 1) / rows_per;
}
__device__ __forceinline__ Place place_of(const AttnArgs& a, uint32_t w, uint32_t grid, int rows_per, AttnSeq& s) {
  const int lane = thread_again() & 63;
  if (a.seqs == 1) {
    s = attn_seq(a, 0);
    const uint32_t tiles = (uint32_t)tiles_of(a, s.nq, rows_per);
    uint32_t t, h;
    if (a.causal) {
      h = w % (uint32_t)a.kv_heads;
      t = w / (uint32_t)a.kv_heads;
    } else {  // blocks of threads go to the 8 XCDs in turn: each gets a run of the heads' tiles
      const uint32_t xcd = w & 7u;
      w = xcd * (grid >> 3) + min(xcd, grid & 7u) + (w >> 3);
      t = w % max(tiles, 1u);
      h = w / max(tiles, 1u);
    }
    if (t >= tiles || h >= (uint32_t)a.kv_heads) return {-1, 0, 0};
    return {0, (int)h, (int)(a.causal ? tiles - 1 - t : t)};
  }
  const int h = (int)(w % (uint32_t)a.kv_heads), t = (int)(w / (uint32_t)a.kv_heads);
  if (a.direct) {
    const int tile = a.direct - 1 - t / a.seqs, b = t % a.seqs;
    s = attn_seq(a, b);
    return {tile >= 0 && tile < tiles_of(a, s.nq, rows_per) ? b : -1, h, tile};
  }
  // A lane has the sequences lane, 64 + lane, ...; tiles of the first EACH of them stay in registers, those of
  // others are worked out again (a block of threads among 1001 sequences takes 3 us to find its rows).
  constexpr int EACH = 16;
  int mine[EACH] = {};
#pragma unroll
  for (int i0 = 0; i0 < EACH; i0 += 4) {
    if (64 * i0 >= a.seqs) break;
    int n[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) n[i] = attn_queries(a, min(64 * (i0 + i) + lane, a.seqs - 1));
#pragma unroll
    for (int i = 0; i < 4; ++i) mine[i0 + i] = 64 * (i0 + i) + lane < a.seqs ? tiles_of(a, n[i], rows_per) : 0;
  }
  const auto sum_over = [&](int level) {  // tiles at levels from `level` on
    int n = 0;
#pragma unroll
    for (int i0 = 0; i0 < EACH; i0 += 4) {
      if (64 * i0 >= a.seqs) break;
#pragma unroll
      for (int i = 0; i < 4; ++i) n += max(mine[i0 + i] - level, 0);
    }
#pragma unroll 4
    for (int b = lane + 64 * EACH; b < a.seqs; b += 64) n += max(tiles_of(a, attn_queries(a, b), rows_per) - level, 0);
    return wave_total(n);
  };
  if (sum_over(0) <= t) return {-1, 0, 0};
  int top = 0;
#pragma unroll
  for (int i = 0; i < EACH; ++i) top = max(top, mine[i]);
#pragma unroll 4
  for (int b = lane + 64 * EACH; b < a.seqs; b += 64) top = max(top, tiles_of(a, attn_queries(a, b), rows_per));
  // the level that holds the t-th tile from the top: from lo on there are more than t, from hi on not
  int lo = 0, hi = wave_top(top), above = 0;  // above: tiles at levels from hi on
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2, n = sum_over(mid);
    if (n > t) lo = mid;
    else hi = mid, above = n;
  }
  int rank = t - above, b = -1;  // among the sequences that reach level lo
  const auto take = [&](int b0, int tiles) {
    if (b >= 0) return;
    uint64_t reach = __ballot(tiles > lo);
    const int n = __builtin_popcountll(reach);
    if (rank < n) {
      for (; rank; --rank) reach &= reach - 1;
      b = b0 + (int)__builtin_ctzll(reach);
    } else {
      rank -= n;
    }
  };
#pragma unroll
  for (int i = 0; i < EACH; ++i) take(64 * i, mine[i]);
  for (int b0 = 64 * EACH; b0 < a.seqs && b < 0; b0 += 64)
    take(b0, b0 + lane < a.seqs ? tiles_of(a, attn_queries(a, b0 + lane), rows_per) : 0);
  if (b < 0) return {-1, 0, 0};
  s = attn_seq(a, b);
  return {b, h, lo};
}

// Four keys of a lane's channel, from four rows of V in LDS.
__device__ __forceinline__ s16x4 read_turned(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

// Channels 4 half + 0..3 of two neighbouring groups of 8, x and y, as bf16: half 0 gets all 8 of x,
// half 1 of y.
__device__ __forceinline__ u32x4 rows_of_8(f32x4 x, f32x4 y) {
  u32x4 w;
#pragma unroll
  for (int e = 0; e < 2; ++e) {
    const auto z = __builtin_amdgcn_permlane32_swap(bf16_pair(x[2 * e], x[2 * e + 1]), bf16_pair(y[2 * e], y[2 * e + 1]), false, false);
    w[e] = z[0];
    w[2 + e] = z[1];
  }
  return w;
}

// ------------------------------------------------------------------ joining parts
// The parts of one tile of rows, in their order. A wave has 32 channels of 32 rows, its lanes what
// they had in the kernel that wrote the parts; (m, l) of all parts are loaded at once, and outputs
// of four parts, as each load waits for memory behind the last-level cache (1.5 us).
template <int D, int ROWS, bool F32>
__global__ __launch_bounds__(256) void attn_many_join_kernel(AttnArgs a) {
  constexpr int ND = D / 32, WAVES = ROWS / 32 * ND;  // of a tile
  const int64_t j = blockIdx.x / (WAVES / 4);
  const int4 join = a.joins[j];
  if (join.w == 0) return;
  const int lane = threadIdx.x & 63, half = lane >> 5, wave = blockIdx.x % (WAVES / 4) * 4 + (threadIdx.x >> 6);
  const int set = wave / ND, d = wave % ND, in_tile = 32 * set + (lane & 31), h = join.y, parts = join.w;
  const AttnSeq sq = attn_seq(a, join.x);
  const int rows = sq.nq * a.group, r = join.z * ROWS + in_tile;
  if (join.z * ROWS + 32 * set >= rows) return;
  const int64_t slot = j * a.splits;
  float2 ml[kMostParts];
  float m = kLowest, l = 0.0f;
#pragma unroll
  for (int i = 0; i < kMostParts; ++i) ml[i] = a.part_ml[(slot + min(i, parts - 1)) * ROWS + in_tile];
#pragma unroll
  for (int i = 0; i < kMostParts; ++i) m = fmaxf(m, ml[i].x);
  const f32x4* const y = reinterpret_cast<const f32x4*>(a.part) + ((slot * (ROWS / 32) + set) * ND + d) * 4 * 64 + lane;
  constexpr int64_t STEP = (int64_t)ROWS * D / 4;  // from part to part
  f32x4 x[4] = {};
#pragma unroll
  for (int i0 = 0; i0 < kMostParts; i0 += 4) {
    if (i0 >= parts) break;
    f32x4 z[4][4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int c = 0; c < 4; ++c) z[i][c] = y[min(i0 + i, parts - 1) * STEP + c * 64];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (i0 + i >= parts) break;
      // In fp32 m follows the values too: the factor of a sum that counts can be under fp32's range, its root is not.
      const float root = F32 ? exp2_fast(0.5f * (ml[i0 + i].x - m)) : 1.0f, f = F32 ? root * root : exp2_fast(ml[i0 + i].x - m);
      l += F32 ? ml[i0 + i].y * root * root : ml[i0 + i].y * f;
#pragma unroll
      for (int c = 0; c < 4; ++c) x[c] += z[i][c] * f;
    }
  }
  const float inv = attn_inverse(l);
  const bool live = r < rows;
  const int query = sq.q0 + r / a.group, hq = h * a.group + r % a.group;
  const int64_t at = (int64_t)query * a.out.st + (int64_t)hq * a.out.sh + 32 * d;
  if constexpr (F32) {
#pragma unroll
    for (int c = 0; c < 4; ++c)
      if (live) *reinterpret_cast<f32x4*>((float*)a.out.data + at + 8 * c + 4 * half) = x[c] * inv;
  } else {
#pragma unroll
    for (int c = 0; c < 4; c += 2) {
      const u32x4 w = rows_of_8(x[c] * inv, x[c + 1] * inv);
      if (live) *reinterpret_cast<u32x4*>((uint16_t*)a.out.data + at + 8 * c + 8 * half) = w;
    }
  }
  if (live && half == 0 && d == 0 && a.lse) a.lse[(int64_t)query * a.q_heads + hq] = attn_lse(m, l);
}

}  // namespace
}  // namespace rc
