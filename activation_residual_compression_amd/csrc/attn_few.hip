// Attention over packed sequences, for few query rows.
//
// One block of threads: 16 rows of one key head of one sequence (row r: query r / G, query
// head h * G + r % G), a part of the keys. Its four waves read steps of 32 keys of their own
// straight into registers and keep their own running maximum and sum; they are joined in
// LDS, and the parts of the keys by the one that is done last.
//
// S^T = K Q^T and O^T = V^T P^T: a lane holds scores of one row only (its column). The
// first product is in the type of the inputs (bf16 or fp32). The second is in fp32 for
// both: its matrix instruction takes one key of 16 channels in a lane, which is how a row
// of V comes from memory, so V needs no transposing, and the weights are not rounded. Scores
// of key 16 t + 4 g + i are result i of tile t in lane group g, and the second product's
// step (t, i) takes key 16 t + 4 g + i from lane group g: no exchange between lanes either.
#include <type_traits>

#include "attn_device.hpp"

namespace rc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));

// E consecutive values, of 8 or 16 bytes, as they lie.
template <int BYTES>
__device__ __forceinline__ auto load_raw(const void* p) {
  if constexpr (BYTES == 8) return *reinterpret_cast<const u32x2*>(p);
  else return *reinterpret_cast<const u32x4*>(p);
}
// Value i of them in fp32.
template <bool F32, typename RAW>
__device__ __forceinline__ float value_of(const RAW& w, int i) {
  if constexpr (F32) return __uint_as_float(w[i]);
  else return i % 2 ? bf16_hi(w[i / 2]) : bf16_lo(w[i / 2]);
}

template <int D, bool F32>
__global__ __launch_bounds__(256, F32 ? 2 : 3) void attn_few_kernel(AttnArgs a) {
  constexpr int NCT = D / 16, VE = F32 ? 4 : D / 16, NB = D / (16 * VE), NK = F32 ? D / 16 : D / 32;
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  typedef typename std::conditional<!F32 && D == 64, u32x2, u32x4>::type VRaw;
  __shared__ float so[4][16][D + 4];
  __shared__ float2 sml[4][16];
  __shared__ bool last;
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x % a.splits, group = blockIdx.x / a.splits;
  const AttnSeq sq = attn_seq(a, b);
  const int rows = sq.nq * a.group, r0 = group * 16, r1 = min(r0 + 16, rows);
  if (r0 >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, quad = lane >> 4;
  const int r = min(r0 + col, r1 - 1);
  const int lim = attn_limit(a, sq, r / a.group);
  const int lim_lo = attn_limit(a, sq, r0 / a.group), lim_hi = attn_limit(a, sq, (r1 - 1) / a.group);
  int parts, from, to;
  if (!attn_part(a, lim_hi, split, parts, from, to)) return;

  // operand s of the first product: channels 32 s + 8 quad + 0..7, in fp32 16 s + 4 quad + 0..3
  u32x4 qr[NK];
  {
    const IO* q = (const IO*)a.q.data + (int64_t)(sq.q0 + r / a.group) * a.q.st + (int64_t)(h * a.group + r % a.group) * a.q.sh;
#pragma unroll
    for (int s = 0; s < NK; ++s) qr[s] = load_raw<16>(q + (F32 ? 16 * s + 4 * quad : 32 * s + 8 * quad));
  }
  const IO* const kh = (const IO*)a.k.data + (int64_t)sq.k0 * a.k.st + (int64_t)h * a.k.sh;
  const IO* const vh = (const IO*)a.v.data + (int64_t)sq.k0 * a.v.st + (int64_t)h * a.v.sh;

  // o[VE * n + e], result jj: channel 16 VE n + VE (4 quad + jj) + e
  f32x4 o[NCT];
#pragma unroll
  for (int d = 0; d < NCT; ++d) o[d] = f32x4{0, 0, 0, 0};
  float m_run = kLowest, l_run = 0.0f;
  for (int j = from + 32 * wave; j < to; j += 128) {
    u32x4 k[2][NK];
    VRaw v[2][4][NB];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const IO* p = kh + (int64_t)min(j + 16 * t + col, sq.nk - 1) * a.k.st;
#pragma unroll
      for (int s = 0; s < NK; ++s) k[t][s] = load_raw<16>(p + (F32 ? 16 * s + 4 * quad : 32 * s + 8 * quad));
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const IO* p = vh + (int64_t)min(j + 16 * t + 4 * quad + i, sq.nk - 1) * a.v.st + VE * col;
#pragma unroll
        for (int n = 0; n < NB; ++n) v[t][i][n] = load_raw<sizeof(VRaw)>(p + 16 * VE * n);
      }
    f32x4 s4[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s4[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        if constexpr (F32) {
#pragma unroll
          for (int i = 0; i < 4; ++i)
            s4[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(k[t][s][i]), __uint_as_float(qr[s][i]), s4[t], 0, 0, 0);
        } else {
          s4[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, k[t][s]), __builtin_bit_cast(bf16x8, qr[s]),
                                                          s4[t], 0, 0, 0);
        }
      }
    }
    // Some row does not see all keys of the step: their scores are replaced, and what is not
    // finite among the values that some row may not see is taken out of the product (zero
    // times it is NaN) and added below for the rows that see it.
    bool strange = false;
    if (j + 32 > lim_lo) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int token = j + 16 * t + 4 * quad + i;
          if (token >= lim) s4[t][i] = -INFINITY;
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < VE; ++e) strange |= token >= lim_lo && not_finite(value_of<F32>(v[t][i][n], e));
        }
      strange = __any(strange);
    }
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s4[t][i]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = max_halves(top);
    const float m_new = fmaxf(m_run, top * a.scale);
    if (__any(m_new > m_run)) {
      const float alpha = exp2_fast(m_run - m_new);
      l_run *= alpha;
#pragma unroll
      for (int d = 0; d < NCT; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] *= alpha;
      m_run = m_new;
    }
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float p = exp2_fast(fmaf(s4[t][i], a.scale, -m_run));
        l_run += p;
        const bool hide = strange && j + 16 * t + 4 * quad + i >= lim_lo;
#pragma unroll
        for (int n = 0; n < NB; ++n)
#pragma unroll
          for (int e = 0; e < VE; ++e) {
            float x = value_of<F32>(v[t][i][n], e);
            if (hide && not_finite(x)) x = 0.0f;
            o[VE * n + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(x, p, o[VE * n + e], 0, 0, 0);
          }
      }
    if (strange) {
      for (int token = max(j, lim_lo); token < min(j + 32, lim); ++token) {
        const IO* p = vh + (int64_t)token * a.v.st;
#pragma unroll
        for (int d = 0; d < NCT; ++d)
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const IO* at = p + 16 * VE * (d / VE) + VE * (4 * quad + i) + d % VE;
            float x;
            if constexpr (F32) x = *at;
            else x = bf16_lo(*at);
            if (not_finite(x)) o[d][i] += x;
          }
      }
    }
  }
  l_run += __shfl_xor(l_run, 16);
  l_run += __shfl_xor(l_run, 32);
#pragma unroll
  for (int d = 0; d < NCT; ++d)
#pragma unroll
    for (int i = 0; i < 4; ++i) so[wave][col][16 * VE * (d / VE) + VE * (4 * quad + i) + d % VE] = o[d][i];
  if (quad == 0) sml[wave][col] = make_float2(m_run, l_run);
  __syncthreads();

  // join the waves: 16 threads a row, D / 16 values each
  const int rr = tid >> 4, d0 = (tid & 15) * NCT;
  const bool mine = r0 + rr < r1;
  float m = kLowest, l = 0.0f, f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) m = fmaxf(m, sml[w][rr].x);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = exp2_fast(sml[w][rr].x - m);
    l += sml[w][rr].y * f[w];
  }
  f32x4 x[NCT / 4];
#pragma unroll
  for (int i = 0; i < NCT / 4; ++i) {
    x[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) x[i] += *reinterpret_cast<const f32x4*>(&so[w][rr][d0 + 4 * i]) * f[w];
  }
  if (parts > 1) {
    // The part that is done last joins them all, in their order, so the result does not
    // depend on which one that was. Partial results pass between XCDs, whose L2 caches are
    // not coherent: they are written and read past them.
    const int64_t all = (int64_t)a.kv_heads * a.q_tokens * a.group;
    const int64_t at = ((int64_t)h * a.q_tokens + sq.q0) * a.group + r0 + rr;
    if (mine) {
#pragma unroll
      for (int i = 0; i < NCT / 4; ++i) {
        put_pair(a.part + (split * all + at) * D + d0 + 4 * i, make_float2(x[i].x, x[i].y));
        put_pair(a.part + (split * all + at) * D + d0 + 4 * i + 2, make_float2(x[i].z, x[i].w));
      }
      if ((tid & 15) == 0) put_pair(&a.part_ml[split * all + at].x, make_float2(m, l));
    }
    uint32_t* arrived = a.arrived + ((int64_t)b * a.kv_heads + h) * (gridDim.x / a.splits) + group;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this thread's stores are done
    __syncthreads();
    if (tid == 0) last = atomicAdd(arrived, 1u) == (uint32_t)parts - 1u;
    __syncthreads();
    if (!last) return;
    if (tid == 0) *arrived = 0;
    if (!mine) return;
    m = kLowest;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < NCT / 4; ++i) x[i] = f32x4{0, 0, 0, 0};
    for (int s = 0; s < parts; ++s) {
      const float2 ml = get_pair(&a.part_ml[s * all + at].x);
      float2 y[NCT / 2];
#pragma unroll
      for (int i = 0; i < NCT / 2; ++i) y[i] = get_pair(a.part + (s * all + at) * D + d0 + 2 * i);
      const float m_new = fmaxf(m, ml.x), fo = exp2_fast(m - m_new), fs = exp2_fast(ml.x - m_new);
      m = m_new;
      l = l * fo + ml.y * fs;
#pragma unroll
      for (int i = 0; i < NCT / 4; ++i)
        x[i] = x[i] * fo + f32x4{y[2 * i].x, y[2 * i].y, y[2 * i + 1].x, y[2 * i + 1].y} * fs;
    }
  }
  if (!mine) return;
  const int query = sq.q0 + (r0 + rr) / a.group, head = h * a.group + (r0 + rr) % a.group;
  const float inv = attn_inverse(l);
  IO* out = (IO*)a.out.data + (int64_t)query * a.out.st + (int64_t)head * a.out.sh + d0;
#pragma unroll
  for (int i = 0; i < NCT / 4; ++i) {
    const f32x4 y = x[i] * inv;
    if constexpr (F32)
      *reinterpret_cast<f32x4*>(out + 4 * i) = y;
    else
      *reinterpret_cast<u32x2*>(out + 4 * i) = u32x2{bf16_pair(y.x, y.y), bf16_pair(y.z, y.w)};
  }
  if (a.lse && (tid & 15) == 0) a.lse[(int64_t)query * a.q_heads + head] = attn_lse(m, l);
}

template <int D, bool F32>
hipError_t run(const AttnArgs& a, hipStream_t s) {
  const int64_t x = (int64_t)a.splits * (((int64_t)a.max_q * a.group + 15) / 16);
  if (x > INT32_MAX) return hipErrorInvalidValue;
  attn_few_kernel<D, F32><<<dim3((unsigned)x, (unsigned)a.kv_heads, (unsigned)a.seqs), 256, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_few(const AttnArgs& a, bool bf16, hipStream_t s) {
  if (a.dim == 64) return bf16 ? run<64, false>(a, s) : run<64, true>(a, s);
  return bf16 ? run<128, false>(a, s) : run<128, true>(a, s);
}

}  // namespace rc
