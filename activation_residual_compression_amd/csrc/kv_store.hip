// Store into the 8-bit key/value cache: quantise, append, mean keys.
//
// One block of threads owns one 64-token block of one key head, of K or of V:
// every scale is the maximum over exactly what one thread block holds, so a
// single pass over the new values is enough (read once, 2 or 4 B an element; one
// byte written). HBM bound for whole sequences (in bf16 each of a thread's loads waits
// for the one before): 4 x 4608 tokens of 24 x 128 bf16 68 to 72 us (5.0 to 4.7 TB/s), 4444
// of 30 x 64 fp32 16 us (5.3). For single tokens the launch and the chain of reads that
// wait for one another (start, table, new values, scale and, of V, earlier codes) are
// what it costs: 16 sequences, 8 heads of 128, 6.1 us, in fp32 6.4.
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

// 4 x 4 bytes, rows to columns: byte i of c[j] is byte j of r[i].
__device__ __forceinline__ void turn4(const uint32_t (&r)[4], uint32_t (&c)[4]) {
  const uint32_t ab_lo = __builtin_amdgcn_perm(r[1], r[0], 0x05010400u), ab_hi = __builtin_amdgcn_perm(r[1], r[0], 0x07030602u);
  const uint32_t cd_lo = __builtin_amdgcn_perm(r[3], r[2], 0x05010400u), cd_hi = __builtin_amdgcn_perm(r[3], r[2], 0x07030602u);
  c[0] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x05040100u);
  c[1] = __builtin_amdgcn_perm(cd_lo, ab_lo, 0x07060302u);
  c[2] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x05040100u);
  c[3] = __builtin_amdgcn_perm(cd_hi, ab_hi, 0x07060302u);
}

// 8 values of a row; once: past the caches. Inputs that fit the last-level cache are
// often still there from what wrote them (a peer's reconstruction of 4444 x 1920 fp32,
// read twice over: 15.7 us against 21.2 past the caches); larger ones only push other
// data out (226 MB of bf16: 68 us past them, 75 through).
template <typename IN, bool ONCE>
__device__ __forceinline__ void row8_in(const IN* p, float (&x)[8]) {
  if constexpr (ONCE) {
    const f32x4 a = load4<IN>(p), b = load4<IN>(p + 4);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = a[i];
      x[4 + i] = b[i];
    }
  } else {
    row8<IN>(p, x);
  }
}

template <int D, typename KIN, typename VIN, bool ONCE>
__global__ __launch_bounds__(256) void kv_store_kernel(KvStoreArgs a) {
  constexpr int ROW = D / 8, TURNS = 64 * ROW / 256;  // threads of a token's row, rows of a thread
  constexpr int LS = D + 16;     // LDS row of codes; 16 B of padding spread the columns over the banks
  constexpr int UNITS = 64 * D / 16 / 256;  // 16-byte units of a thread
  constexpr int QUADS = D / 4, PARTS = 256 / QUADS;
  __shared__ uint32_t wave_max[4];
  __shared__ __align__(16) uint8_t codes[64 * LS];
  __shared__ __align__(16) float sums[PARTS][D];
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
  const int64_t row = kv_row(g, block, head);
  uint8_t* base = (is_v ? g.v : g.k) + row * (64 * D);
  const int tid = threadIdx.x;

  float x[TURNS][8];
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int t = tid / ROW + 256 / ROW * i, c0 = tid % ROW * 8;
#pragma unroll
    for (int u = 0; u < 8; ++u) x[i][u] = 0.0f;
    if (t >= first && t < last) {
      const int64_t tok = t0 + t - start;
      if (is_v)
        row8_in<VIN, ONCE>((const VIN*)a.v.data + b * a.v.sb + tok * a.v.st + head * a.v.sh + c0, x[i]);
      else
        row8_in<KIN, ONCE>((const KIN*)a.k.data + b * a.k.sb + tok * a.k.st + head * a.k.sh + c0, x[i]);
    }
  }
  // K's earlier codes, as units of the layout [D/16][64][16]
  u32x4 was[UNITS];
  if (begun && !is_v) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u)
      if ((tid & 63) < first) was[u] = *reinterpret_cast<const u32x4*>(base + (tid + 256 * u) * 16);
  }
#pragma unroll
  for (int i = 0; i < TURNS; ++i)
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const uint32_t v = __float_as_uint(x[i][u]) & 0x7FFFFFFFu;
      top = max(top, v < 0x7F800000u ? v : 0u);
    }
  top = group_max_u32<32>(top);
  top = max(top, (uint32_t)__shfl_xor((int)top, 32));
  if ((tid & 63) == 0) wave_max[tid >> 6] = top;
  float* scale = (is_v ? g.v_scale : g.k_scale) + row;
  const int e_was = begun ? scale_exponent(*scale) : kKvEMin;
  __syncthreads();
  top = max(max(wave_max[0], wave_max[1]), max(wave_max[2], wave_max[3]));
  const int e = begun ? max(exponent_for(top), e_was) : exponent_for(top);
  const bool again = begun && e > e_was;
  const float inv = pow2f(-e), down = pow2f(e_was - e);

#pragma unroll
  for (int i = 0; i < TURNS; ++i) {
    const int t = tid / ROW + 256 / ROW * i, c0 = tid % ROW * 8;
    if (t >= first)
      *reinterpret_cast<u32x2*>(codes + t * LS + c0) = u32x2{encode4(x[i][0], x[i][1], x[i][2], x[i][3], inv),
                                                             encode4(x[i][4], x[i][5], x[i][6], x[i][7], inv)};
  }
  if (begun && !is_v && (tid & 63) < first) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      if (again) {
#pragma unroll
        for (int i = 0; i < 4; ++i) was[u][i] = recode4(was[u][i], down);
      }
      *reinterpret_cast<u32x4*>(codes + (tid & 63) * LS + ((tid + 256 * u) >> 6) * 16) = was[u];
    }
  }
  __syncthreads();

  if (!is_v) {
    const int t = tid & 63;
    if (!begun || (t >= first && t < last) || (again && t < first)) {
#pragma unroll
      for (int u = 0; u < UNITS; ++u)
        *reinterpret_cast<u32x4*>(base + (tid + 256 * u) * 16) =
            *reinterpret_cast<const u32x4*>(codes + t * LS + ((tid + 256 * u) >> 6) * 16);
    }
    // mean key: sums of at most 64 codes are whole multiples of 2^-9 below 2^15, exact in
    // fp32 in any order
    const int quad = tid % QUADS, part = tid / QUADS;
    f32x4 s = {0, 0, 0, 0};
#pragma unroll 2
    for (int i = part * (64 / PARTS); i < (part + 1) * (64 / PARTS); ++i) {
      uint32_t w = *reinterpret_cast<const uint32_t*>(codes + i * LS + 4 * quad);
      if (i >= last) w = 0;
      const f32x4 c = {__builtin_amdgcn_cvt_f32_fp8(w, 0), __builtin_amdgcn_cvt_f32_fp8(w, 1),
                       __builtin_amdgcn_cvt_f32_fp8(w, 2), __builtin_amdgcn_cvt_f32_fp8(w, 3)};
#pragma unroll
      for (int k = 0; k < 4; ++k) s[k] += c[k] == c[k] ? c[k] : 0.0f;  // NaN counts as 0
    }
    *reinterpret_cast<f32x4*>(&sums[part][4 * quad]) = s;
    __syncthreads();
    if (tid < 64) {
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int p = 0; p < PARTS; ++p) {
        s0 += sums[p][tid];
        if (D == 128) s1 += sums[p][tid + D / 2];
      }
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
    // V: a unit is 16 tokens of one channel, layout [4][D][16]: the codes turn, 4 channels
    // and 16 tokens a thread
    if (tid == 0) *scale = pow2f(e);
    if (!begun) {
      if (tid >= D) return;
      const int lo = tid / QUADS * 16, c0 = tid % QUADS * 4;
      uint32_t out[4][4];  // [channel][4 tokens]
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        uint32_t r[4], c[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) r[i] = *reinterpret_cast<const uint32_t*>(codes + (lo + 4 * q + i) * LS + c0);
        turn4(r, c);
#pragma unroll
        for (int k = 0; k < 4; ++k) out[k][q] = c[k];
      }
      u32x4* at = reinterpret_cast<u32x4*>(base + (lo / 16 * D + c0) * 16);
#pragma unroll
      for (int k = 0; k < 4; ++k) at[k] = u32x4{out[k][0], out[k][1], out[k][2], out[k][3]};
      return;
    }
    // beside earlier tokens: only the units that change, one a thread
    for (int unit = tid; unit < 4 * D; unit += 256) {
      const int lo = unit / D * 16, d = unit % D;
      const bool any_new = lo < last && lo + 16 > first;
      if (!any_new && !(again && lo < first)) continue;
      u32x4* at = reinterpret_cast<u32x4*>(base + unit * 16);
      u32x4 out = *at;
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
      *at = out;
    }
  }
}

template <int D, typename KIN, typename VIN>
hipError_t run(const KvStoreArgs& a, hipStream_t s) {
  const dim3 grid((unsigned)((a.tokens + 63) / 64 + 1), (unsigned)(2 * a.g.kv_heads), (unsigned)a.g.batch);
  if (a.once)
    kv_store_kernel<D, KIN, VIN, true><<<grid, 256, 0, s>>>(a);
  else
    kv_store_kernel<D, KIN, VIN, false><<<grid, 256, 0, s>>>(a);
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
