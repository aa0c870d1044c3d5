// The join of attentions over different tokens.
//
// out = sum_i w_i out_i / sum_i w_i with w_i = 2^((lse_i - m) log2 e), m the largest lse; lse
// = m + log(sum_i w_i). 16 bytes of a row to a lane, every part read once: HBM bound. A lane
// reads all that it needs before it writes, and a row's lanes are of one wave, so the
// output may lie where a part does.
#include "attn_device.hpp"

namespace rc {
namespace {

// Values of a lane: 4, or 8 where inputs are bf16.
template <int D, bool IN16, bool OUT16>
__global__ __launch_bounds__(256) void attn_join_kernel(AttnJoinArgs a) {
  constexpr int E = IN16 ? 8 : 4, LANES = D / E;
  constexpr float kLog2e = 1.44269504088896340736f;
  const int64_t row = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int d0 = threadIdx.x % LANES * E;
  if (row >= a.rows) return;
  const int h = (int)(row % a.heads);
  const int64_t bt = row / a.heads;
  const int t = (int)(bt % a.tokens);
  const int64_t b = bt / a.tokens;
  float lse[RC_ATTN_MAX_PARTS], x[RC_ATTN_MAX_PARTS][E], m = -INFINITY;
#pragma unroll
  for (int i = 0; i < RC_ATTN_MAX_PARTS; ++i) {
    if (i >= a.parts) break;
    lse[i] = a.lses[i][row];
    const int64_t at = b * a.in[i].sb + (int64_t)t * a.in[i].st + (int64_t)h * a.in[i].sh + d0;
    if constexpr (IN16) {
      row8<uint16_t>((const uint16_t*)a.in[i].data + at, x[i]);
    } else {
      const f32x4 w = *reinterpret_cast<const f32x4*>((const float*)a.in[i].data + at);
#pragma unroll
      for (int e = 0; e < 4; ++e) x[i][e] = w[e];
    }
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
    if constexpr (OUT16)
      *reinterpret_cast<u32x2*>((uint16_t*)a.out.data + at + e) = u32x2{bf16_pair(y[e], y[e + 1]), bf16_pair(y[e + 2], y[e + 3])};
    else
      *reinterpret_cast<f32x4*>((float*)a.out.data + at + e) = f32x4{y[e], y[e + 1], y[e + 2], y[e + 3]};
  }
  if (a.lse && d0 == 0) a.lse[row] = total == 0.0f ? -INFINITY : m + logf(total);
}

template <int D, bool IN16, bool OUT16>
hipError_t run(const AttnJoinArgs& a, hipStream_t s) {
  constexpr int64_t per = 256 / (D / (IN16 ? 8 : 4));
  const int64_t grid = (a.rows + per - 1) / per;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  attn_join_kernel<D, IN16, OUT16><<<(unsigned)grid, 256, 0, s>>>(a);
  return hipGetLastError();
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
