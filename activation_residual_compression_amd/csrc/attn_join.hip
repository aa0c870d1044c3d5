// The join of attentions over different tokens.
//
// out = sum_i w_i out_i / sum_i w_i with w_i = 2^((lse_i - m) log2 e), m the largest lse; lse
// = m + log(sum_i w_i). 16 bytes of a row to a lane, every part read once: HBM bound. A lane
// reads all that it needs before it writes, and a row's lanes are of one wave, so the
// output may lie where a part does. 4444 tokens, 30 heads of 64, four fp32 parts (173 MB):
// 29.2 us from HBM, 5.9 TB/s.
#include "attn_device.hpp"

namespace rc {
namespace {

template <bool FAR, typename T>
__device__ __forceinline__ T load_16(const void* p) {
  if constexpr (FAR) return __builtin_nontemporal_load(reinterpret_cast<const T*>(p));
  else return *reinterpret_cast<const T*>(p);
}

// Values of a lane: 4, or 8 where inputs are bf16. FAR: the data is more than the caches hold, and passes them
// (29.2 us for the call above, through them 33.9; the same tensors again and again 28.2 and 25.5).
template <int D, bool IN16, bool OUT16, bool FAR>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnJoinArgs a, int64_t first) {
  constexpr int E = IN16 ? 8 : 4, LANES = D / E;
  constexpr float kLog2e = 1.44269504088896340736f;
  // Blocks of threads go to the 8 XCDs in turn; each gets a run of the rows.
  const uint32_t runs = gridDim.x / 8, w = blockIdx.x < 8 * runs ? blockIdx.x % 8 * runs + blockIdx.x / 8 : blockIdx.x;
  const int64_t row = (first + w) * (256 / LANES) + threadIdx.x / LANES;
  const int d0 = threadIdx.x % LANES * E;
  if (row >= a.rows) return;
  int h, t;
  int64_t b;
  if (a.rows >> 32 == 0) {  // divisions of 64 bits take as long as all else
    const uint32_t bt = (uint32_t)row / (uint32_t)a.heads;
    h = (int)((uint32_t)row - bt * (uint32_t)a.heads);
    b = bt / (uint32_t)a.tokens;
    t = (int)(bt - (uint32_t)b * (uint32_t)a.tokens);
  } else {
    const int64_t bt = row / a.heads;
    h = (int)(row % a.heads);
    b = bt / a.tokens;
    t = (int)(bt % a.tokens);
  }
  float lse[RC_ATTN_MAX_PARTS], x[RC_ATTN_MAX_PARTS][E], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < RC_ATTN_MAX_PARTS; ++i) {
    if (i >= a.parts) break;
    lse[i] = a.lses[i][row];
    const int64_t at = b * a.in[i].sb + (int64_t)t * a.in[i].st + (int64_t)h * a.in[i].sh + d0;
    if constexpr (IN16) {
      const u32x4 v = load_16<FAR, u32x4>((const uint16_t*)a.in[i].data + at);
#pragma unroll
      for (int e = 0; e < E; ++e) x[i][e] = e % 2 ? bf16_hi(v[e / 2]) : bf16_lo(v[e / 2]);
    } else {
      const f32x4 v = load_16<FAR, f32x4>((const float*)a.in[i].data + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = v[e];
    }
  }
#pragma unroll
  for (int i = 0; i < RC_ATTN_MAX_PARTS; ++i) {  // when all loads are on their way
    if (i >= a.parts) break;
    m = fmaxf(m, lse[i]);
  }
  float total = 0.0f, y[E];
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] = 0.0f;
#pragma unroll
  for (int i = 0; i < RC_ATTN_MAX_PARTS; ++i) {
    if (i >= a.parts) break;
    if (lse[i] == -INFINITY) continue;
    const float w = exp2_fast((lse[i] - m) * kLog2e);
    total += w;
#pragma unroll
    for (int e = 0; e < E; ++e) y[e] = fmaf(w, x[i][e], y[e]);
  }
  const float inv = attn_inverse(total);
#pragma unroll
  for (int e = 0; e < E; ++e) y[e] *= inv;
  const int64_t at = b * a.out.sb + (int64_t)t * a.out.st + (int64_t)h * a.out.sh + d0;
#pragma unroll
  for (int e = 0; e < E; e += 4) {
    if constexpr (OUT16) {
      const u32x2 v = {bf16_pair(y[e], y[e + 1]), bf16_pair(y[e + 2], y[e + 3])};
      u32x2* to = reinterpret_cast<u32x2*>((uint16_t*)a.out.data + at + e);
      if constexpr (FAR) __builtin_nontemporal_store(v, to);
      else *to = v;
    } else {
      const f32x4 v = {y[e], y[e + 1], y[e + 2], y[e + 3]};
      f32x4* to = reinterpret_cast<f32x4*>((float*)a.out.data + at + e);
      if constexpr (FAR) __builtin_nontemporal_store(v, to);
      else *to = v;
    }
  }
  if (a.lse && d0 == 0) a.lse[row] = total == 0.0f ? -INFINITY : m + logf(total);
}

template <int D, bool IN16, bool OUT16>
hipError_t run(const AttnJoinArgs& a, hipStream_t s) {
  constexpr int64_t per = 256 / (D / (IN16 ? 8 : 4));
  const int64_t grid = (a.rows + per - 1) / per;
  const bool far = a.rows * a.parts * D * (IN16 ? 2 : 4) > (int64_t)128 << 20;
  return launch_all(grid, [&](int64_t first, unsigned blocks) {
    if (far) attn_join_kernel<D, IN16, OUT16, true><<<blocks, 256, 0, s>>>(a, first);
    else attn_join_kernel<D, IN16, OUT16, false><<<blocks, 256, 0, s>>>(a, first);
  });
}

template <int D>
hipError_t pick(const AttnJoinArgs& a, bool in16, bool out16, hipStream_t s) {
  if (in16) return out16 ? run<D, true, true>(a, s) : run<D, true, false>(a, s);
  return out16 ? run<D, false, true>(a, s) : run<D, false, false>(a, s);
}

}  // namespace

hipError_t launch_attn_join(const AttnJoinArgs& a, bool in_bf16, bool out_bf16, hipStream_t s) {
  return a.dim == 64 ? pick<64>(a, in_bf16, out_bf16, s) : pick<128>(a, in_bf16, out_bf16, s);
}

}  // namespace rc
