// Store into the 8-bit key/value cache: quantise, append, mean keys.
//
// One block of threads owns one 64-token block of one key head, of K or of V:
// every scale is the maximum over exactly what one thread block holds, so a
// single pass over the new values is enough (read once, 2 or 4 B an element; one
// byte written). HBM bound for whole sequences; for single tokens the launch and
// one dependent read (start, table, codes) are what it costs.
#include "kv_device.hpp"

namespace rc {
namespace {

// x * 2^-e -> clamped, for the e4m3 conversion (round to nearest even; NaN stays).
__device__ __forceinline__ float fit(float x, float inv) {
  const float y = x * inv;
  return fabsf(y) > 448.0f ? copysignf(448.0f, y) : y;
}
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d, float inv) {
  uint32_t w = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fit(a, inv), fit(b, inv), 0, false);
  return (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(fit(c, inv), fit(d, inv), (int)w, true);
}
// Codes of an earlier scale rounded again in a larger one (down = 2^(old - new)).
__device__ __forceinline__ uint32_t recode4(uint32_t w, float down) {
  return encode4(__builtin_amdgcn_cvt_f32_fp8(w, 0), __builtin_amdgcn_cvt_f32_fp8(w, 1),
                 __builtin_amdgcn_cvt_f32_fp8(w, 2), __builtin_amdgcn_cvt_f32_fp8(w, 3), down);
}
__device__ __forceinline__ float value_of(uint32_t byte) { return __builtin_amdgcn_cvt_f32_fp8(byte, 0); }

// Smallest e with amax <= 448 * 2^e = 1.75 * 2^(e + 8), in the allowed range.
__device__ __forceinline__ int exponent_for(uint32_t amax_bits) {
  const int e = (int)(amax_bits >> 23) - 135 + ((amax_bits & 0x7FFFFFu) > 0x600000u ? 1 : 0);
  return min(max(e, kKvEMin), kKvEMax);
}

template <int D, typename KIN, typename VIN>
__global__ __launch_bounds__(256) void kv_store_kernel(KvStoreArgs a) {
  constexpr int W = D / 4;       // values of a thread: a quarter of a token's row
  constexpr int LS = D + 16;     // LDS row of codes; 16 B of padding spread the columns over the banks
  __shared__ uint32_t wave_max[4];
  __shared__ __align__(16) uint8_t codes[64 * LS];
  __shared__ float sums[2][D];
  const KvGeom& g = a.g;
  const int b = blockIdx.z, head = blockIdx.y >> 1;
  const bool is_v = blockIdx.y & 1;
  const int64_t start = a.start[b];
  if (start < 0) return;
  const int n = a.count ? min(max(a.count[b], 0), a.tokens) : a.tokens;
  const int64_t j64 = start / 64 + blockIdx.x;
  if (j64 >= g.seq_blocks || j64 * 64 >= start + n) return;
  const int block = kv_block(g, b, (int)j64);
  if (block < 0) return;
  const int64_t t0 = j64 * 64;
  const int first = start > t0 ? (int)(start - t0) : 0;              // slots before: earlier tokens
  const int last = start + n < t0 + 64 ? (int)(start + n - t0) : 64;  // slots from here on: none
  const bool begun = first > 0;

  const int tid = threadIdx.x, t = tid >> 2, c0 = (tid & 3) * W;
  const bool is_new = t >= first && t < last;
  float x[W];
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = 0.0f;
  if (is_new) {
    const int64_t tok = t0 + t - start;
#pragma unroll
    for (int i = 0; i < W; i += 8) {
      float y[8];
      if (is_v)
        row8<VIN>((const VIN*)a.v.data + b * a.v.sb + tok * a.v.st + head * a.v.sh + c0 + i, y);
      else
        row8<KIN>((const KIN*)a.k.data + b * a.k.sb + tok * a.k.st + head * a.k.sh + c0 + i, y);
#pragma unroll
      for (int u = 0; u < 8; ++u) x[i + u] = y[u];
    }
  }
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    const uint32_t u = __float_as_uint(x[i]) & 0x7FFFFFFFu;
    top = max(top, u < 0x7F800000u ? u : 0u);
  }
  top = group_max_u32<32>(top);
  top = max(top, (uint32_t)__shfl_xor((int)top, 32));
  if ((tid & 63) == 0) wave_max[tid >> 6] = top;
  __syncthreads();
  top = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));

  const int64_t row = kv_row(g, block, head);
  float* scale = (is_v ? g.v_scale : g.k_scale) + row;
  const int e_was = begun ? scale_exponent(*scale) : kKvEMin;
  const int e = begun ? max(exponent_for(top), e_was) : exponent_for(top);
  const bool again = begun && e > e_was;
  const float inv = pow2f(-e), down = pow2f(e_was - e);
  uint8_t* base = (is_v ? g.v : g.k) + row * (64 * D);

  uint32_t w[W / 4];
#pragma unroll
  for (int i = 0; i < W / 4; ++i) w[i] = encode4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3], inv);

  if (!is_v) {
    // K: a thread's values are 16-byte units of the layout [D/16][64][16]
#pragma unroll
    for (int u = 0; u < W / 16; ++u) {
      u32x4* unit = reinterpret_cast<u32x4*>(base + ((c0 / 16 + u) * 64 + t) * 16);
      if (t < first) {
        const u32x4 was = *unit;
        w[4 * u] = was.x; w[4 * u + 1] = was.y; w[4 * u + 2] = was.z; w[4 * u + 3] = was.w;
        if (again) {
#pragma unroll
          for (int i = 0; i < 4; ++i) w[4 * u + i] = recode4(w[4 * u + i], down);
        }
      }
      if (!begun || is_new || (again && t < first))
        *unit = u32x4{w[4 * u], w[4 * u + 1], w[4 * u + 2], w[4 * u + 3]};
    }
  }
#pragma unroll
  for (int i = 0; i < W / 4; ++i) *reinterpret_cast<uint32_t*>(codes + t * LS + c0 + 4 * i) = w[i];
  __syncthreads();

  if (!is_v) {
    // mean key: sums of at most 64 codes are whole multiples of 2^-9 below 2^15, exact in fp32
    constexpr int PARTS = 256 / D, SPAN = 64 / PARTS;
    const int d = tid % D, part = tid / D;
    float s = 0.0f;
    for (int i = part * SPAN; i < min(last, (part + 1) * SPAN); ++i) {
      const float c = value_of(codes[i * LS + d]);
      s += c == c ? c : 0.0f;  // NaN counts as 0
    }
    if constexpr (PARTS == 4) {
      // D = 64: a wave holds one part; fold the four by way of LDS in two steps
      if (part >= 2) sums[part - 2][d] = s;
      __syncthreads();
      if (part < 2) s += sums[part][d];
      __syncthreads();
    }
    if (part == 1) sums[1][d] = s;
    __syncthreads();
    if (part == 0) sums[0][d] = s + sums[1][d];
    __syncthreads();
    if (tid < 64) {
      const float s0 = sums[0][tid], s1 = D == 128 ? sums[0][tid + D / 2] : 0.0f;
      uint32_t m = max(__float_as_uint(s0) & 0x7FFFFFFFu, __float_as_uint(s1) & 0x7FFFFFFFu);
      m = group_max_u32<32>(m);
      m = max(m, (uint32_t)__shfl_xor((int)m, 32));
      const float amax = __uint_as_float(m);
      const float up = amax > 0.0f ? 127.0f * (1.0f / amax) : 0.0f;
      int8_t* mean = g.k_mean + row * D;
      mean[tid] = (int8_t)(int)rintf(s0 * up);
      if (D == 128) mean[tid + D / 2] = (int8_t)(int)rintf(s1 * up);
      if (tid == 0) {
        g.k_mean_scale[row] = amax / (float)(127 * last) * pow2f(e);
        *scale = pow2f(e);
      }
    }
  } else {
    // V: a unit is 16 tokens of one channel, layout [4][D][16]: the codes turn in LDS
    if (tid == 0) *scale = pow2f(e);
    for (int unit = tid; unit < 4 * D; unit += 256) {
      const int gq = unit / D, d = unit % D, lo = 16 * gq;
      const bool any_new = lo < last && lo + 16 > first;
      if (begun && !any_new && !(again && lo < first)) continue;
      u32x4* at = reinterpret_cast<u32x4*>(base + (gq * D + d) * 16);
      const bool need = begun && (lo < first || lo + 16 > last);
      const u32x4 was = need ? *at : u32x4{0, 0, 0, 0};
      uint32_t out[4] = {was.x, was.y, was.z, was.w};
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const uint32_t re = again ? recode4(out[q], down) : out[q];
        uint32_t r = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int tok = lo + 4 * q + i;
          uint32_t byte = (tok < first ? re : out[q]) >> (8 * i) & 255u;
          if (tok >= first && tok < last) byte = codes[tok * LS + d];
          r |= byte << (8 * i);
        }
        out[q] = r;
      }
      *at = u32x4{out[0], out[1], out[2], out[3]};
    }
  }
}

template <int D, typename KIN, typename VIN>
hipError_t run(const KvStoreArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + 63) / 64 + 1), (unsigned)(2 * a.g.kv_heads), (unsigned)a.g.batch);
  kv_store_kernel<D, KIN, VIN><<<grid, 256, 0, s>>>(a);
  return hipGetLastError();
}
template <int D>
hipError_t pick(const KvStoreArgs& a, bool kb, bool vb, hipStream_t s) {
  if (kb) return vb ? run<D, uint16_t, uint16_t>(a, s) : run<D, uint16_t, float>(a, s);
  return vb ? run<D, float, uint16_t>(a, s) : run<D, float, float>(a, s);
}

}  // namespace

hipError_t launch_kv_store(const KvStoreArgs& a, bool k_bf16, bool v_bf16, hipStream_t s) {
  return a.g.dim == 64 ? pick<64>(a, k_bf16, v_bf16, s) : pick<128>(a, k_bf16, v_bf16, s);
}

}  // namespace rc
