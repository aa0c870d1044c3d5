// Choice of blocks by a cheap score: 8-bit query times 8-bit mean key.
//
// The products are whole numbers (at most 127^2 * 128 < 2^21), so the score is
// the same whatever the order of the sums, and the choice is exactly
// reproducible; two fp32 roundings (times the mean's scale, times the query's
// largest value) are part of its definition. One block of threads scores all
// blocks for one tile of queries of one key head (v_mfma_i32_32x32x32_i8, mean
// keys as rows, queries as columns), then picks the k best by a radix select on
// the scores' bits in LDS.
#include "kv_device.hpp"

namespace rc {
namespace {

constexpr int kRows = 128;               // query rows that are in LDS at a time
constexpr uint32_t kNone = 0x007FFFFFu;  // key of -infinity: seen by no query

// Order-preserving map of fp32 to u32.
__device__ __forceinline__ uint32_t sort_key(float x) {
  const uint32_t u = __float_as_uint(x);
  return u >> 31 ? ~u : u | 0x80000000u;
}

template <int D, typename IN>
__global__ __launch_bounds__(256) void kv_select_kernel(KvAttendArgs a) {
  constexpr int QS = D + 16;  // LDS row of query codes
  extern __shared__ uint32_t keys[];
  __shared__ __align__(16) uint8_t qc[kRows * QS];
  __shared__ float qs[kRows];
  __shared__ int qlim[kRows];
  __shared__ uint32_t hist[256];
  __shared__ uint32_t pick[2];
  const KvGeom& g = a.g;
  const int b = blockIdx.z, h = blockIdx.y, tile = blockIdx.x, G = g.group;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, l32 = lane & 31, half = lane >> 5;
  const int len = kv_length(a, b);
  const int q0 = tile * a.q_tile, rows = min(a.q_tile, a.queries - q0) * G;
  const int lim_lo = kv_limit(a, len, q0), lim_hi = kv_limit(a, len, q0 + rows / G - 1);
  const int nb = (lim_hi + 63) / 64;
  for (int j = tid; j < nb; j += 256) keys[j] = 0;

  for (int r0 = 0; r0 < rows; r0 += kRows) {
    __syncthreads();
    {
      const int r = tid >> 1, c0 = (tid & 1) * (D / 2);
      const bool live = r0 + r < rows;
      const int i = q0 + (r0 + r) / G, hq = h * G + (r0 + r) % G;
      float x[D / 2];
      float top = 0.0f;
#pragma unroll
      for (int c = 0; c < D / 2; c += 8) {
        float y[8] = {0, 0, 0, 0, 0, 0, 0, 0};
        if (live) row8<IN>((const IN*)a.q.data + b * a.q.sb + (int64_t)i * a.q.st + hq * a.q.sh + c0 + c, y);
#pragma unroll
        for (int u = 0; u < 8; ++u) {
          x[c + u] = y[u];
          top = fmaxf(top, fabsf(y[u]));
        }
      }
      top = fmaxf(top, dpp_f32<kQuadXor1>(top));
      const float up = top > 0.0f ? 127.0f * (1.0f / top) : 0.0f;
#pragma unroll
      for (int c = 0; c < D / 2; c += 4) {
        uint32_t w = 0;
#pragma unroll
        for (int u = 0; u < 4; ++u) w |= ((uint32_t)(int)rintf(x[c + u] * up) & 255u) << (8 * u);
        *reinterpret_cast<uint32_t*>(qc + r * QS + c0 + c) = w;
      }
      if ((tid & 1) == 0) {
        qs[r] = top;
        qlim[r] = live ? kv_limit(a, len, i) : 0;
      }
    }
    __syncthreads();
    const int cols = min(rows - r0, kRows);
    for (int bt = wave * 32; bt < nb; bt += 128) {
      const int j = bt + l32;
      const int block = j < nb ? kv_block(g, b, j) : -1;
      const int64_t row = block < 0 ? 0 : kv_row(g, block, h);
      i32x4 m[D / 32];
#pragma unroll
      for (int s = 0; s < D / 32; ++s)
        m[s] = block < 0 ? i32x4{0, 0, 0, 0}
                         : *reinterpret_cast<const i32x4*>(g.k_mean + row * D + s * 32 + half * 16);
      const float ks = block < 0 ? 0.0f : g.k_mean_scale[row];
      float best[16], ksr[16];
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        best[i] = -INFINITY;
        ksr[i] = __shfl(ks, 8 * (i / 4) + 4 * half + i % 4);
      }
      for (int ct = 0; ct < cols; ct += 32) {
        i32x16 acc = {};
#pragma unroll
        for (int s = 0; s < D / 32; ++s) {
          const i32x4 q = *reinterpret_cast<const i32x4*>(qc + (ct + l32) * QS + s * 32 + half * 16);
          acc = __builtin_amdgcn_mfma_i32_32x32x32_i8(m[s], q, acc, 0, 0, 0);
        }
        const float mul = qs[ct + l32];
        const int seen = (qlim[ct + l32] + 63) / 64 - bt;  // rows below: blocks whose first token is seen
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float v = (float)acc[i] * ksr[i] * mul + 0.0f;  // + 0: -0 and 0 tie
          if (8 * (i / 4) + 4 * half + i % 4 < seen) best[i] = fmaxf(best[i], v);
        }
      }
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float v = group_max<32>(best[i]);
        const int jj = bt + 8 * (i / 4) + 4 * half + i % 4;
        if (l32 == i && jj < nb) keys[jj] = max(keys[jj], sort_key(v));
      }
    }
  }
  __syncthreads();
  const int own0 = (max(lim_lo, 1) - 1) / 64;
  for (int j = tid; j < nb; j += 256) {
    uint32_t k = keys[j];
    if (a.causal && j >= own0) k = 0xFFFFFFFFu;
    if (kv_block(g, b, j) < 0) k = 0;
    keys[j] = k;
  }
  // radix select: the key of the keep-th best, and how many of that key are taken
  uint32_t prefix = 0, want = (uint32_t)a.keep;
  for (int shift = 24; shift >= 0; shift -= 8) {
    hist[tid] = 0;
    __syncthreads();
    for (int j = tid; j < nb; j += 256) {
      const uint32_t k = keys[j];
      if (k > kNone && (shift == 24 || k >> (shift + 8) == prefix)) atomicAdd(&hist[k >> shift & 255u], 1u);
    }
    __syncthreads();
    if (wave == 0) {
      uint32_t c[4], sum = 0;
#pragma unroll
      for (int i = 0; i < 4; ++i) sum += c[i] = hist[4 * lane + i];
      uint32_t above = sum;  // entries in this lane's bins and the higher ones
#pragma unroll
      for (int d = 1; d < 64; d <<= 1) {
        const uint32_t o = (uint32_t)__shfl_down((int)above, d);
        if (lane + d < 64) above += o;
      }
      uint32_t higher = above - sum;
      if (lane == 0 && above < want) {  // fewer than wanted: take all
        pick[0] = 0;
        pick[1] = 0xFFFFFFFFu;
      }
      if (above >= want && higher < want) {
#pragma unroll
        for (int i = 3; i >= 0; --i) {
          if (higher < want && higher + c[i] >= want) {
            pick[0] = 4 * lane + i;
            pick[1] = want - higher;
          }
          higher += c[i];
        }
      }
    }
    __syncthreads();
    if (pick[1] == 0xFFFFFFFFu) break;  // only at the first digit: later ones hold at least `want`
    prefix = prefix << 8 | pick[0];
    want = pick[1];
    __syncthreads();
  }
  const bool all = pick[1] == 0xFFFFFFFFu;
  if (wave == 0) {
    int32_t* out = a.blocks_out + (((int64_t)b * g.kv_heads + h) * a.tiles + tile) * a.keep;
    int n = 0;
    uint32_t ties = 0;
    const uint64_t below = ((uint64_t)1 << lane) - 1;
    for (int j0 = 0; j0 < nb; j0 += 64) {
      const int j = j0 + lane;
      const uint32_t k = j < nb ? keys[j] : 0;
      const bool ok = k > kNone;
      const bool tie = ok && !all && k == prefix;
      const uint64_t tied = __ballot(tie);
      const bool take = ok && (all || k > prefix || (tie && ties + __popcll(tied & below) < want));
      const uint64_t taken = __ballot(take);
      if (take) out[n + __popcll(taken & below)] = j;
      n += __popcll(taken);
      ties += __popcll(tied);
    }
    for (int i = n + lane; i < a.keep; i += 64) out[i] = -1;
  }
}

template <int D, typename IN>
hipError_t run(const KvAttendArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)a.tiles, (unsigned)a.g.kv_heads, (unsigned)a.g.batch);
  kv_select_kernel<D, IN><<<grid, 256, (size_t)((a.max_len + 63) / 64) * 4, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_kv_select(const KvAttendArgs& a, bool bf16, hipStream_t s) {
  if (a.g.dim == 64) return bf16 ? run<64, uint16_t>(a, s) : run<64, float>(a, s);
  return bf16 ? run<128, uint16_t>(a, s) : run<128, float>(a, s);
}

}  // namespace rc
