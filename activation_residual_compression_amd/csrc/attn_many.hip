// Attention over packed sequences, for many query rows, bf16.
//
// One block of threads: 4 waves of 32 U rows each of one key head of one sequence (row r:
// query r / G, query head h * G + r % G), a part of the keys. Tiles of 64 keys and values go
// through three LDS buffers that all waves share, one barrier a tile.
//
// S^T = K Q^T and O^T = V^T P^T: a lane holds scores of one row only (its column), the softmax
// is in the lane, and its weights, rounded to bf16, are the second product's operand as they
// are: result i of the first lies at key 8 (i / 4) + 4 half + i % 4, so lane half `half` holds
// keys 16 m + 4 half + 0..3 and 16 m + 8 + 4 half + 0..3 for step m of the second product, and V
// is read in that order, transposed four keys at a time by the LDS's own transposing read.
//
// Softmax in base 2, p = 2^(S c - m). m is not the running maximum: it is raised only when the
// weights of a step sum to more than 2^10, which the sum shows that is needed anyway, so the
// accumulators are rescaled a few times in all, and no maximum is taken otherwise. bf16 and
// fp32 hold such weights as well as those up to 1; both cancel in out = O / l.
#include <algorithm>

#include "attn_device.hpp"

namespace rc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef short s16x4 __attribute__((ext_vector_type(4)));

constexpr float kMost = 0x1p10f;
constexpr int kTile = 64;

// A tile in LDS: rows of 2 D bytes without gaps, as the loads that write them lay them. The
// 16-byte chunks of a row are in the order c ^ turn(row), so that a column of chunks (K, 16
// rows a step of a read) or four rows of 32 bytes (V) meet different banks.
template <int D>
__device__ __forceinline__ int k_turn(int row) { return D == 128 ? row & 15 : row >> 1 & 7; }
template <int D>
__device__ __forceinline__ int v_turn(int row) { return D == 128 ? (row & 7) << 1 : (row >> 1 & 3) << 1; }

// 16 bytes a lane from memory into LDS at `to` (one for the wave) + 16 lane, past the
// registers, from base + offset or from an address of each lane. The compiler's own form of this
// makes every later read of LDS wait for it; here the wait is the caller's (vmcnt), once a tile.
// Nothing else in these kernels uses m0.
__device__ __forceinline__ void load_lds(uint32_t to, uint32_t offset, const void* base) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"s"(to), "v"(offset), "s"(base) : "memory");
}
__device__ __forceinline__ void load_lds(uint32_t to, const void* at) {
  asm volatile("s_mov_b32 m0, %0\n\ts_nop 0\n\tglobal_load_lds_dwordx4 %1, off" ::"s"(to), "v"(at) : "memory");
}

// Which rows a block of threads does. Tiles of rows are given out by their number from the
// end of their sequence, highest first over all sequences: with a causal mask the long ones
// first, and without it those of the long sequences.
struct Place {
  int b, h, tile;  // b < 0: none
};
__device__ __forceinline__ int tiles_of(const AttnArgs& a, int b, int rows_per) {
  return (attn_seq(a, b).nq * a.group + rows_per - 1) / rows_per;
}
__device__ __forceinline__ int wave_sum(int x) {
#pragma unroll
  for (int d = 32; d; d /= 2) x += __shfl_xor(x, d);
  return x;
}
__device__ __forceinline__ int wave_max(int x) {
#pragma unroll
  for (int d = 32; d; d /= 2) x = max(x, __shfl_xor(x, d));
  return x;
}
__device__ __forceinline__ Place place_of(const AttnArgs& a, uint32_t w, uint32_t grid, int rows_per) {
  const int lane = threadIdx.x & 63;
  if (a.seqs == 1) {
    const uint32_t tiles = (uint32_t)tiles_of(a, 0, rows_per);
    uint32_t t, h;
    if (a.causal) {
      h = w % (uint32_t)a.kv_heads;
      t = w / (uint32_t)a.kv_heads;
    } else {  // blocks of threads go to the 8 XCDs in turn: each gets a run of the heads' tiles
      const uint32_t xcd = w & 7u;
      w = xcd * (grid >> 3) + min(xcd, grid & 7u) + (w >> 3);
      t = w % tiles;
      h = w / tiles;
    }
    if (t >= tiles || h >= (uint32_t)a.kv_heads) return {-1, 0, 0};
    return {0, (int)h, (int)(a.causal ? tiles - 1 - t : t)};
  }
  const int h = (int)(w % (uint32_t)a.kv_heads), t = (int)(w / (uint32_t)a.kv_heads);
  // the level (number of a tile in its sequence) that holds the t-th tile from the top
  int top = 0;
  for (int b = lane; b < a.seqs; b += 64) top = max(top, tiles_of(a, b, rows_per));
  int lo = 0, hi = wave_max(top);  // tiles at levels from lo on: more than t; from hi on: not
  int above = 0;                   // tiles at levels from hi on
  {
    int n = 0;
    for (int b = lane; b < a.seqs; b += 64) n += tiles_of(a, b, rows_per);
    if (wave_sum(n) <= t) return {-1, 0, 0};
  }
  while (hi - lo > 1) {
    const int mid = (lo + hi) / 2;
    int n = 0;
    for (int b = lane; b < a.seqs; b += 64) n += max(tiles_of(a, b, rows_per) - mid, 0);
    n = wave_sum(n);
    if (n > t) lo = mid;
    else hi = mid, above = n;
  }
  int rank = t - above;  // among the sequences that reach level lo
  for (int b0 = 0; b0 < a.seqs; b0 += 64) {
    const int b = b0 + lane;
    uint64_t reach = __ballot(b < a.seqs && tiles_of(a, min(b, a.seqs - 1), rows_per) > lo);
    const int n = __builtin_popcountll(reach);
    if (rank < n) {
      for (; rank; --rank) reach &= reach - 1;
      return {b0 + (int)__builtin_ctzll(reach), h, lo};
    }
    rank -= n;
  }
  return {-1, 0, 0};
}

// Four keys of a lane's channel, from four rows of V in LDS.
__device__ __forceinline__ s16x4 read_turned(const char* p) {
  return __builtin_amdgcn_ds_read_tr16_b64_v4i16((__attribute__((address_space(3))) s16x4*)p);
}

template <int D, int U>
__global__ __launch_bounds__(256, 2) void attn_many_kernel(AttnArgs a) {
  constexpr int NK = D / 16, ND = D / 32, ROWS = 128 * U;
  constexpr int PER = D / 8, ROW = 2 * D, HALF = kTile * ROW, BYTES = 2 * HALF;  // chunks, bytes of a row; bytes of K, of a tile
  constexpr int C = D / 32, STEP = kTile / C;  // loads of a thread for a tile of K, and the rows between two of them
  __shared__ __align__(1024) char shared[2 * BYTES];
  __shared__ int strange;  // the last tile that held a value which is not finite and hidden from some row
  const Place place = place_of(a, blockIdx.x, gridDim.x, ROWS);
  const int b = __builtin_amdgcn_readfirstlane(place.b), h = __builtin_amdgcn_readfirstlane(place.h);
  if (b < 0) return;
  AttnSeq sq = attn_seq(a, b);
  sq = {__builtin_amdgcn_readfirstlane(sq.q0), __builtin_amdgcn_readfirstlane(sq.nq), __builtin_amdgcn_readfirstlane(sq.k0),
        __builtin_amdgcn_readfirstlane(sq.nk)};
  const int rows = sq.nq * a.group, r0 = __builtin_amdgcn_readfirstlane(place.tile) * ROWS;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 31, half = lane >> 5;
  const int lim_lo = attn_limit(a, sq, r0 / a.group);
  const int lim_hi = attn_limit(a, sq, (min(r0 + ROWS, rows) - 1) / a.group);
  const int tiles = (lim_hi + kTile - 1) / kTile;
  if (tid == 0) strange = -1;

  // staging: load i of a thread has chunk lane % PER of row STEP i + srow, whose turn does not depend on i
  const char* const kh = (const char*)((const uint16_t*)a.k.data + (int64_t)sq.k0 * a.k.st + (int64_t)h * a.k.sh);
  const char* const vh = (const char*)((const uint16_t*)a.v.data + (int64_t)sq.k0 * a.v.st + (int64_t)h * a.v.sh);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)shared;
  const bool near = (a.k.st | a.v.st) < (int64_t)1 << 24;  // a tile's offsets fit 32 bits
  const auto stage = [&](int tile) {
    int again = threadIdx.x;  // what follows from it would take registers through the loop
    asm volatile("" : "+v"(again));
    const int lane = again & 63, srow = wave * (STEP / 4) + lane / PER;
    const uint32_t k_turned = (uint32_t)((lane % PER) ^ k_turn<D>(srow)) * 16, v_turned = (uint32_t)((lane % PER) ^ v_turn<D>(srow)) * 16;
    const uint32_t to = lds0 + (uint32_t)((tile & 1) * BYTES + wave * (STEP / 4) * ROW);
    if (near && (tile + 1) * kTile <= sq.nk) {
      const uint32_t k_off = (uint32_t)srow * (uint32_t)(2 * a.k.st) + k_turned, v_off = (uint32_t)srow * (uint32_t)(2 * a.v.st) + v_turned;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        load_lds(to + i * STEP * ROW, k_off, kh + (int64_t)(tile * kTile + i * STEP) * (2 * a.k.st));
        load_lds(to + HALF + i * STEP * ROW, v_off, vh + (int64_t)(tile * kTile + i * STEP) * (2 * a.v.st));
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < C; ++i) {
        const int64_t token = min(tile * kTile + i * STEP + srow, sq.nk - 1);
        load_lds(to + i * STEP * ROW, kh + token * (2 * a.k.st) + k_turned);
        load_lds(to + HALF + i * STEP * ROW, vh + token * (2 * a.v.st) + v_turned);
      }
    }
  };
  if (tiles > 0) stage(0);

  // rows of this wave, and its queries: operand f has channels 16 f + 8 half + 0..7
  bf16x8 q[U][NK];
  float m_run[U], l_run[U];
  int wave_lo = INT32_MAX, wave_hi = 0;  // what its rows see
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 32 * U * wave + 32 * u + col, rr = min(r, rows - 1);
    const uint16_t* p = (const uint16_t*)a.q.data + (int64_t)(sq.q0 + rr / a.group) * a.q.st + (int64_t)(h * a.group + rr % a.group) * a.q.sh;
#pragma unroll
    for (int f = 0; f < NK; ++f) q[u][f] = *reinterpret_cast<const bf16x8*>(p + 16 * f + 8 * half);
    m_run[u] = kLowest;
    l_run[u] = 0.0f;
  }
  {
    const int first = r0 + 32 * U * wave, last = min(first + 32 * U, rows) - 1;
    if (first < rows) {
      wave_lo = attn_limit(a, sq, first / a.group);
      wave_hi = attn_limit(a, sq, last / a.group);
    }
  }
  const int my_tiles = (wave_hi + kTile - 1) / kTile;
  const auto limit = [&](int u) {  // keys that the lane's row sees
    int again = threadIdx.x;
    asm volatile("" : "+v"(again));
    return attn_limit(a, sq, min(r0 + 32 * U * wave + 32 * u + (again & 31), rows - 1) / a.group);
  };
  f32x16 o[U][ND];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int d = 0; d < ND; ++d) o[u][d] = f32x16{};

  // places of the operands in a tile: row part + (chunk part ^ 32 f), (^ 64 d)
  const int vrow = 4 * half + (lane & 15) / 4;
  int k_at = col * ROW + (half ^ k_turn<D>(col)) * 16;
  int v_at = HALF + vrow * ROW + ((2 * (lane >> 4 & 1) + (lane & 3) / 2) ^ v_turn<D>(vrow)) * 16 + (lane & 1) * 8;

  for (int t = 0; t < tiles; ++t) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this wave's loads of tile t are in LDS
    __syncthreads();                                  // the others' too, and tile t - 1 is read
    if (t + 1 < tiles) stage(t + 1);
    char* const tile = shared + (t & 1) * BYTES;
    if ((t + 1) * kTile > lim_lo) {
      // What is not finite among values that some row does not see is taken out of the product
      // (zero times it is NaN) and added after it for the rows that see it.
      int again = threadIdx.x;
      asm volatile("" : "+v"(again));
      const int lane = again & 63, srow = wave * (STEP / 4) + lane / PER;
      bool odd = false;
#pragma unroll 1
      for (int i = 0; i < C; ++i) {
        const int row = i * STEP + srow;
        u32x4* at = reinterpret_cast<u32x4*>(tile + HALF + row * ROW + lane % PER * 16);
        u32x4 x = *at;
        bool here = false;
#pragma unroll
        for (int w = 0; w < 4; ++w) {
          const bool lo = (x[w] & 0x7F80u) == 0x7F80u, hi = (x[w] & 0x7F800000u) == 0x7F800000u;
          here |= lo || hi;
          x[w] &= (lo ? 0u : 0xFFFFu) | (hi ? 0u : 0xFFFF0000u);
        }
        if (here && t * kTile + row >= lim_lo) {
          *at = x;
          odd = true;
        }
      }
      if (odd) strange = t;
      __syncthreads();
    }
    if (t >= my_tiles) continue;
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {
      const int first = t * kTile + 32 * hb;  // key
      asm volatile("" : "+v"(k_at), "+v"(v_at));  // or all their forms would be kept in registers
      f32x16 s[U] = {};
      {
        const auto key = [&](int f) { return *reinterpret_cast<const bf16x8*>(tile + hb * 32 * ROW + (k_at ^ 32 * f)); };
        bf16x8 kf = key(0);
#pragma unroll
        for (int f = 0; f < NK; ++f) {
          const bf16x8 now = kf;
          if (f + 1 < NK) kf = key(f + 1);
#pragma unroll
          for (int u = 0; u < U; ++u) s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now, q[u][f], s[u], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
      if (first + 32 > wave_lo) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // by bits, not by comparisons, whose 32 results at once would spill scalars
          const int left = min(max(limit(u) - first - 4 * half, 0), 31);  // the last bit, key 28, is the highest used
          const uint32_t seen = (1u << left) - 1u;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t on = (uint32_t)((int32_t)(seen << (31 - 8 * (i / 4) - i % 4)) >> 31);
            s[u][i] = __uint_as_float((__float_as_uint(s[u][i]) & on) | (0xFF800000u & ~on));
          }
        }
      }
      u32x4 ph[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const auto weigh = [&](float& sum) {
          sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {  // four at a time, so that they take few registers
            float p[4];
#pragma unroll
            for (int e = 0; e < 4; ++e) p[e] = exp2_fast(fmaf(s[u][i + e], a.scale, -m_run[u]));
#pragma unroll
            for (int e = 0; e < 4; ++e) sum += p[e];
            ph[u][i / 8][i % 8 / 2] = bf16_pair(p[0], p[1]);
            ph[u][i / 8][i % 8 / 2 + 1] = bf16_pair(p[2], p[3]);
            __builtin_amdgcn_sched_barrier(0);
          }
        };
        float sum;
        weigh(sum);
        if (__any(sum > kMost)) {
          float top = s[u][0];
#pragma unroll
          for (int i = 1; i < 16; ++i) top = fmaxf(top, s[u][i]);
          const float m_new = fmaxf(m_run[u], max_halves(top) * a.scale), alpha = exp2_fast(m_run[u] - m_new);
          l_run[u] *= alpha;
          m_run[u] = m_new;
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[u][d][i] *= alpha;
          weigh(sum);
        }
        l_run[u] += sum;
      }
      {
        const auto value = [&](int at) {  // operand at % 2 of channels 32 (at / 2)
          const char* v = tile + (32 * hb + 16 * (at % 2)) * ROW + (v_at ^ 64 * (at / 2));
          return __builtin_bit_cast(bf16x8, __builtin_shufflevector(read_turned(v), read_turned(v + 8 * ROW), 0, 1, 2, 3, 4, 5, 6, 7));
        };
        bf16x8 vf = value(0);
#pragma unroll
        for (int at = 0; at < 2 * ND; ++at) {
          const bf16x8 now = vf;
          if (at + 1 < 2 * ND) vf = value(at + 1);
#pragma unroll
          for (int u = 0; u < U; ++u)
            o[u][at / 2] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now, __builtin_bit_cast(bf16x8, ph[u][at % 2]), o[u][at / 2], 0, 0, 0);
          __builtin_amdgcn_sched_barrier(0);
        }
      }
    }
    if (strange == t) {
      int again = threadIdx.x;
      asm volatile("" : "+v"(again));
      const int half = again >> 5 & 1;
      int lim[U];
#pragma unroll
      for (int u = 0; u < U; ++u) lim[u] = limit(u);
      for (int token = max(t * kTile, lim_lo); token < min((t + 1) * kTile, lim_hi); ++token) {
        const uint16_t* p = (const uint16_t*)(vh + token * (2 * a.v.st));
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int c = 0; c < 4; ++c) {
            const u32x2 w = *reinterpret_cast<const u32x2*>(p + 32 * d + 8 * c + 4 * half);
#pragma unroll
            for (int e = 0; e < 4; ++e) {
              const float y = e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
              const float add = not_finite(y) ? y : 0.0f;
#pragma unroll
              for (int u = 0; u < U; ++u) o[u][d][4 * c + e] += token < lim[u] ? add : 0.0f;
            }
            __builtin_amdgcn_sched_barrier(0);
          }
      }
    }
  }

  // the thread's place again, from its number alone: kept through the loop it would take registers
  int again = threadIdx.x;
  asm volatile("" : "+v"(again));
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int col = again & 31, half = again >> 5 & 1;
    const int r = r0 + 32 * U * wave + 32 * u + col;
    const float l = l_run[u] + __shfl_xor(l_run[u], 32);
    const float inv = attn_inverse(l);
    const int query = sq.q0 + r / a.group, head = h * a.group + r % a.group;
    uint16_t* out = (uint16_t*)a.out.data + (int64_t)query * a.out.st + (int64_t)head * a.out.sh;
    const bool live = r < rows;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int c = 0; c < 2; ++c) {
        // this half has channels 4 half + 0..3 of groups of 8; after the exchange whole groups
        u32x4 w;
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          const uint32_t x = bf16_pair(o[u][d][8 * c + 2 * e] * inv, o[u][d][8 * c + 2 * e + 1] * inv);
          const uint32_t y = bf16_pair(o[u][d][8 * c + 4 + 2 * e] * inv, o[u][d][8 * c + 4 + 2 * e + 1] * inv);
          const auto z = __builtin_amdgcn_permlane32_swap(x, y, false, false);
          w[e] = z[0];
          w[2 + e] = z[1];
        }
        if (live) *reinterpret_cast<u32x4*>(out + 32 * d + 16 * c + 8 * half) = w;
      }
    if (live && half == 0 && a.lse) a.lse[(int64_t)query * a.q_heads + head] = attn_lse(m_run[u], l);
  }
}

template <int D, int U>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  // as many tiles of rows as the sequences can have: they end in the middle of one each
  const int64_t rows = (int64_t)a.q_tokens * a.group, per = 128 * U;
  const int64_t tiles = std::min(rows / per + a.seqs, a.seqs * (((int64_t)a.max_q * a.group + per - 1) / per));
  const int64_t grid = tiles * a.kv_heads;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  attn_many_kernel<D, U><<<(unsigned)grid, 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_many(const AttnArgs& a, int u, hipStream_t s) {
  if (a.dim == 64) return u == 1 ? run<64, 1>(a, s) : run<64, 2>(a, s);
  return u == 1 ? run<128, 1>(a, s) : run<128, 2>(a, s);
}

}  // namespace rc
