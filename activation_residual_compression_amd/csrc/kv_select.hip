// Choice of blocks by a cheap score: 8-bit query times 8-bit mean key.
//
// The products are whole numbers (at most 127^2 * 128 < 2^21), so the score is
// the same whatever the order of the sums, and the choice is exactly
// reproducible; two fp32 roundings (times the mean's scale, times the query's
// largest value) are part of its definition. One block of threads scores all
// blocks for one tile of queries of one key head (v_mfma_i32_32x32x32_i8, mean
// keys as rows, queries as columns), then picks the k best by a radix select on
// the scores' bits in LDS. Bound by latency and by waves without work: the chain of reads
// (length, queries, table, means), in bf16 a thread's query loads, each of which waits for
// the one before, and four digits of the select; waves take 64 blocks at a time, so 125
// blocks leave two of four without any. Measured: 32 of up to 1024 blocks for 8 sequences
// and 8 key heads 13.6 us (either type); 70 of 278 for 35 tiles of 30 heads 30 us (vector
// units 80 % busy); 24 of 125 for 16 tiles of 4 x 128 fp32 rows, 4 heads, 2 sequences 34 us.
#include "kv_device.hpp"

namespace rc {
namespace {

constexpr int kRows = 128;               // query rows that are in LDS at a time
constexpr uint32_t kNone = 0;            // a block that is not there; any score's key is larger

// Order-preserving map of fp32 to u32; that of -infinity, the lowest, is 0x007FFFFF.
__device__ __forceinline__ uint32_t sort_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

// x rounded to a whole number, 0 for a NaN (of a NaN in a query, or of an infinity, whose
// factor is 0): what the instruction gives, and C++'s conversion leaves undefined.
__device__ __forceinline__ int whole(float x) {
  int i;
  asm("v_cvt_i32_f32 %0, %1" : "=v"(i) : "v"(rintf(x)));
  return i;
}

// From a lane and the one that CTRL pairs it with (they differ in the bit that `high`
// tells): the larger of the two values of the half of the registers that the lane keeps.
template <int N, int CTRL>
__device__ __forceinline__ void max_halve(float (&r)[16], bool high) {
#pragma unroll
  for (int i = 0; i < N / 2; ++i) {
    const float keep = high ? r[i + N / 2] : r[i], send = high ? r[i] : r[i + N / 2];
    r[i] = fmaxf(keep, dpp_f32<CTRL>(send));
  }
}
// Maxima over 32 lanes of 16 registers: lane l gets that of register
// 8 * bit 4 + 4 * bit 3 + 2 * bit 2 + bit 1 of l.
__device__ __forceinline__ float max_rows(float (&r)[16], int l) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const auto x = __builtin_amdgcn_permlane16_swap(__float_as_uint(r[i]), __float_as_uint(r[i + 8]), false, false);
    r[i] = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
  }
  constexpr int kRowRor8 = 0x128;
  max_halve<8, kRowRor8>(r, l & 8);
  max_halve<4, kHalfMirror>(r, l & 4);
  max_halve<2, kQuadXor2>(r, l & 2);
  return fmaxf(r[0], dpp_f32<kQuadXor1>(r[0]));
}

// Inclusive sum over the lanes up to this one.
template <int CTRL, int ROWS>
__device__ __forceinline__ uint32_t add_from(uint32_t v) {
  return v + (uint32_t)__builtin_amdgcn_update_dpp(0, (int)v, CTRL, ROWS, 0xF, false);
}
__device__ __forceinline__ uint32_t sum_up_to(uint32_t v) {
  v = add_from<0x111, 0xF>(v);  // from the lane 1, 2, 4, 8 below in the row of 16
  v = add_from<0x112, 0xF>(v);
  v = add_from<0x114, 0xF>(v);
  v = add_from<0x118, 0xF>(v);
  v = add_from<0x142, 0xA>(v);  // the last lane of row 0 to row 1, of row 2 to row 3
  return add_from<0x143, 0xC>(v);  // lane 31 to rows 2 and 3
}

template <int D, typename IN, int WAVES>
__global__ __launch_bounds__(64 * WAVES) void kv_select_kernel(KvAttendArgs a) {
  constexpr int QS = D + 16;  // LDS row of query codes
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) uint8_t qc[kRows * QS];
  __shared__ float qs[kRows];
  __shared__ int qlim[kRows];
  constexpr int THREADS = 64 * WAVES;
  __shared__ uint32_t hist[4][256];
  __shared__ int2 count[WAVES];
  __shared__ __align__(16) float ks[WAVES][64];
  const KvGeom& g = a.g;
  const int b = blockIdx.z, h = blockIdx.y, tile = blockIdx.x, G = g.group;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l32 = lane & 31, half = lane >> 5;
  const int len = kv_length(a, b);
  const int q0 = tile * a.q_tile, rows = min(a.q_tile, a.queries - q0) * G;
  const int lim_lo = kv_limit(a, len, q0), lim_hi = kv_limit(a, len, q0 + rows / G - 1);
  const int nb = (lim_hi + 63) / 64;
  for (int j = tid; j < nb; j += THREADS) keys[j] = kNone;
  for (int i = tid; i < 4 * 256; i += THREADS) (&hist[0][0])[i] = 0;

  for (int r0 = 0; r0 < rows; r0 += kRows) {
    __syncthreads();
    {
      constexpr int TPR = THREADS / kRows, N = D / TPR;  // threads of a row, values of each
      const int r = tid / TPR, c0 = tid % TPR * N;
      const bool live = r0 + r < rows;
      const int i = q0 + (r0 + r) / G, hq = h * G + (r0 + r) % G;
      float x[N];
      float top = 0.0f;
#pragma unroll
      for (int c = 0; c < N; c += 8) {
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (live) row8<IN>((const IN*)a.q.data + b * a.q.sb + (int64_t)i * a.q.st + hq * a.q.sh + c0 + c, y);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          x[c + u] = y[u];
          top = fmaxf(top, fabsf(y[u]));
        }
      }
      top = group_max<TPR>(top);
      float up = 127.0f * (1.0f / top);
      if (!(up < INFINITY)) up = 0.0f;  // a row of zeros, or of less than 2^-121
#pragma unroll
      for (int c = 0; c < N; c += 4) {
        uint32_t w = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) w |= ((uint32_t)whole(x[c + u] * up) & 255u) << (8 * u);
        *reinterpret_cast<uint32_t*>(qc + r * QS + c0 + c) = w;
      }
      if (tid % TPR == 0) {
        qs[r] = top;
        qlim[r] = live ? kv_limit(a, len, i) : 0;
      }
    }
    __syncthreads();
    const int cols = min(rows - r0, kRows);
    for (int b64 = wave * 64; b64 < nb; b64 += THREADS) {
      // two tiles of 32 blocks, all their loads first. No maximum takes a NaN, so a score that
      // is one counts as -infinity. A query of the tile sees each block below nb, so one that
      // exists has a key and can be chosen, whatever its scores; one that does not gets none.
      const int mine = b64 + lane < nb ? kv_block(g, b, b64 + lane) : -1;
      i32x4 mean[2][D / 32];
      ks[wave][lane] = mine < 0 ? 0.0f : g.k_mean_scale[kv_row(g, mine, h)];
      const uint64_t exist = __ballot(mine >= 0);
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int block = __shfl(mine, 32 * u + l32);
        const int64_t row = kv_row(g, max(block, 0), h);
#pragma unroll
        for (int s = 0; s < D / 32; ++s)
          mean[u][s] = *reinterpret_cast<const i32x4*>(g.k_mean + row * D + s * 32 + half * 16);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int bt = b64 + 32 * u;
        if (bt >= nb) break;
        float best[16];  // register i: block bt + 8 (i / 4) + 4 half + i % 4
        f32x4 scale[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) scale[i] = *reinterpret_cast<const f32x4*>(&ks[wave][32 * u + 8 * i + 4 * half]);
#pragma unroll
        for (int i = 0; i < 16; ++i) best[i] = -INFINITY;
        for (int ct = 0; ct < cols; ct += 32) {
          i32x16 acc = {};
#pragma unroll
          for (int s = 0; s < D / 32; ++s) {
            const i32x4 q = *reinterpret_cast<const i32x4*>(qc + (ct + l32) * QS + s * 32 + half * 16);
            acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(mean[u][s], q, acc, 0, 0, 0);
          }
          const float mul = qs[ct + l32];
          const int seen = (qlim[ct + l32] + 63) / 64 - bt;  // blocks of the tile whose first token is seen
          const bool some = __any(seen < 32);
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            float v = (float)acc[i] * scale[i / 4][i % 4] * mul + 0.0f;  // + 0: -0 and 0 tie
            if (some && 8 * (i / 4) + 4 * half + i % 4 >= seen) v = -INFINITY;
            best[i] = fmaxf(best[i], v);
          }
        }
        const float v = max_rows(best, l32);
        const int jj = bt + 8 * (l32 >> 3) + 4 * half + (l32 >> 1 & 3);
        if ((l32 & 1) == 0 && jj < nb && (exist >> (jj - b64) & 1)) keys[jj] = max(keys[jj], sort_key(v));
      }
    }
  }
  __syncthreads();
  const int own0 = (max(lim_lo, 1) - 1) / 64;
  for (int j = tid; j < nb; j += THREADS) {
    if (a.causal && j >= own0 && keys[j] > kNone) keys[j] = 0xFFFFFFFFu;
  }
  __syncthreads();
  // radix select: the key of the keep-th best, and how many of that key are taken. Every
  // wave works out each digit for itself, so a digit costs one barrier.
  uint32_t prefix = 0, want = (uint32_t)a.keep;
  bool all = false;
  for (int digit = 0; digit < 4; ++digit) {
    const int shift = 24 - 8 * digit;
    for (int j = tid; j < nb; j += THREADS) {
      const uint32_t k = keys[j];
      if (k > kNone && (digit == 0 || k >> (shift + 8) == prefix)) atomicAdd(&hist[digit][k >> shift & 255u], 1u);
    }
    __syncthreads();
    // lane l: bins 255 - 4 l and the three below it
    const uint4 bins = *reinterpret_cast<const uint4*>(&hist[digit][252 - 4 * lane]);
    const uint32_t c[4] = {bins.w, bins.z, bins.y, bins.x}, sum = bins.x + bins.y + bins.z + bins.w;
    const uint32_t up_to = sum_up_to(sum);  // entries in this lane's bins and the higher ones
    if ((uint32_t)__builtin_amdgcn_readlane((int)up_to, 63) < want) {  // only at the first digit
      all = true;
      break;
    }
    const int at = __builtin_ctzll(__ballot(up_to >= want));
    uint32_t higher = up_to - sum, bin = 0, rest = 0;
    bool found = false;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (!found && higher + c[i] >= want) {
        found = true;
        bin = 255u - 4u * (uint32_t)lane - (uint32_t)i;
        rest = want - higher;
      }
      higher += c[i];
    }
    prefix = prefix << 8 | (uint32_t)__builtin_amdgcn_readlane((int)bin, at);
    want = (uint32_t)__builtin_amdgcn_readlane((int)rest, at);
  }
  // the taken ones in order: each wave has a run of blocks, and first counts
  const int run = ((nb + WAVES - 1) / WAVES + 63) & ~63, j_end = min((wave + 1) * run, nb);
  int over = 0, ties = 0;
  for (int j0 = wave * run; j0 < j_end; j0 += 64) {
    const uint32_t k = j0 + lane < j_end ? keys[j0 + lane] : 0;
    over += __popcll(__ballot(k > kNone && (all || k > prefix)));
    ties += __popcll(__ballot(k > kNone && !all && k == prefix));
  }
  if (lane == 0) count[wave] = make_int2(over, ties);
  __syncthreads();
  int n = 0, tied = 0;
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    const int2 c = count[w];
    if (w < wave) {
      n += c.x;
      tied += c.y;
    }
    over = w == 0 ? c.x : over + c.x;
    ties = w == 0 ? c.y : ties + c.y;
  }
  n += min(tied, (int)want);
  int32_t* out = a.blocks_out + (((int64_t)b * g.kv_heads + h) * a.tiles + tile) * a.keep;
  const uint64_t below = ((uint64_t)1 << lane) - 1;
  for (int j0 = wave * run; j0 < j_end; j0 += 64) {
    const uint32_t k = j0 + lane < j_end ? keys[j0 + lane] : 0;
    const bool tie = k > kNone && !all && k == prefix;
    const uint64_t same = __ballot(tie);
    const bool take = k > kNone && (all || k > prefix || (tie && tied + __popcll(same & below) < (int)want));
    const uint64_t taken = __ballot(take);
    if (take) out[n + __popcll(taken & below)] = j0 + lane;
    n += __popcll(taken);
    tied += __popcll(same);
  }
  for (int i = over + min(ties, (int)want) + tid; i < a.keep; i += THREADS) out[i] = -1;
}

// 8 waves score the blocks of a tile where the CUs hold all tiles at once that way (one each
// at 128 channels, two at 64, whose registers fit twice) and 4 waves would take more than
// one turn (64 blocks a wave). Measured in us, 4 and 8 waves, single tokens of 8 key heads:
// 128 channels, 256 tiles of 313 blocks 10.9 and 9.0, of 625 14.1 and 11.2; 288 tiles 12.2
// and 15.8, 16.7 and 20.2; 512 12.3 and 16.2, 19.5 and 25.1. 64 channels, 512 tiles of 625
// blocks 17.8 and 16.7, 576 19.3 and 23.8. With 64 blocks or 256, where the rule takes 4:
// 256 tiles 8.0 and 7.3, 8.8 and 8.2 at 128 channels, 512 tiles 7.3 and 8.3, 8.4 and 9.1 at 64.
template <int D, typename IN>
hipError_t run(const KvAttendArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.tiles, (unsigned)a.g.kv_heads, (unsigned)a.g.batch);
  const int blocks = (a.max_len + 63) / 64;
  if ((int64_t)a.tiles * a.g.kv_heads * a.g.batch <= (D == 64 ? 512 : 256) && blocks > 256)
    kv_select_kernel<D, IN, 8><<<grid, 512, (size_t)blocks * 4, s>>>(a);
  else
    kv_select_kernel<D, IN, 4><<<grid, 256, (size_t)blocks * 4, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_select(const KvAttendArgs& a, bool bf16, hipStream_t s) {
  if (a.g.dim == 64) return bf16 ? run<64, uint16_t>(a, s) : run<64, float>(a, s);
  return bf16 ? run<128, uint16_t>(a, s) : run<128, float>(a, s);
}

}  // namespace rc
