// Attention over packed sequences, for few query rows.
//
// One block of threads: 16 rows of one key head of one sequence (row r: query r / G, query
// head h * G + r % G), a part of the keys. Its waves read steps of 32 keys of their own
// straight into registers and keep their own running maximum and sum; they are joined in
// LDS, and the parts of the keys by the block of threads that is done last.
//
// S^T = K Q^T and O^T = V^T P^T: a lane holds scores of one row only (its column), those of
// keys 16 t + 4 g + i as result i of tile t in lane group g. A lane reads D / 16 channels of
// just those 8 keys of V, so that for each channel it holds the operand that the second
// product needs, its row 8 keys of a channel, in the order of the weights: no exchange between
// lanes, and V needs no transposing but that of bytes in a lane. In bf16 the weights enter as
// two bf16 each (16 bits), which costs 16 matrix instructions of 16 cycles a step; in fp32
// both products are in fp32.
//
// Bound by HBM for long keys (one token of 64 sequences of 4000, 32 heads of 128 on 8: 181 us, 5.8
// TB/s; of 65536 tokens 58 us, 4.6 TB/s, the same again and again 50, in fp32 99; 8 ragged ones of up to
// 32768 82 us, 4.7), by the chain of reads for short ones (333 tokens, 24 heads: 8.1 us; 2048 tokens, 32
// heads on 8: 9.4).
// Blocks of threads of one piece and all key heads follow each other: their rows lie next to each
// other in memory (65536 tokens with the pieces of a head after each other: 54 us).
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

// Sum over the lanes up to and with this one.
__device__ __forceinline__ int sum_up_to(int x) {
  x += __builtin_amdgcn_update_dpp(0, x, 0x111, 0xF, 0xF, true);   // from 1, 2, 4, 8 lanes before in the row of 16
  x += __builtin_amdgcn_update_dpp(0, x, 0x112, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x114, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x118, 0xF, 0xF, true);
  x += __builtin_amdgcn_update_dpp(0, x, 0x142, 0xA, 0xF, false);  // the last of a row to the next, for rows 1 and 3
  x += __builtin_amdgcn_update_dpp(0, x, 0x143, 0xC, 0xF, false);  // lane 31 to rows 2 and 3
  return x;
}

// Sequence, group of 16 rows and part that piece `w` of a key head is; called by a whole wave. b < 0: none.
struct Piece {
  int b, group, split, most;  // most: parts that a group has at most
};
__device__ __forceinline__ Piece piece_of(const AttnArgs& a, int w, int groups, AttnSeq& s) {
  const int lane = threadIdx.x & 63;
  if (a.seqs == 1 || a.direct) {
    const int b = a.seqs == 1 ? 0 : w / groups, at = a.seqs == 1 ? w : w % groups;
    s = attn_seq(a, b);
    return {b, at / a.splits, at % a.splits, a.splits};
  }
  // With several parts, or bounds far above the lengths, the pieces are numbered without gaps, sequence by
  // sequence, so that blocks of threads that have work are spread evenly. Offsets that descend may claim more
  // pieces than there are blocks of threads: each group then has one part.
  const auto count = [&](int b0, int most, int& parts) {  // pieces of the lane's sequence
    s = attn_seq(a, min(b0 + lane, a.seqs - 1));
    parts = min(max((s.nk + a.chunk - 1) / a.chunk, 1), most);
    return b0 + lane < a.seqs ? (s.nq * a.group + 15) / 16 * parts : 0;
  };
  int most = a.splits, parts, end = 0;
  if (a.seqs > 64) {
    int64_t all = 0;
#pragma unroll 4
    for (int b0 = 0; b0 < a.seqs; b0 += 64) all += __builtin_amdgcn_readlane(sum_up_to(count(b0, most, parts)), 63);
    if (all > gridDim.x / a.kv_heads) most = 1;
  }
  for (int b0 = 0; b0 < a.seqs; b0 += 64) {
    int mine = count(b0, most, parts);
    end = sum_up_to(mine);
    if (a.seqs <= 64 && __builtin_amdgcn_readlane(end, 63) > (int)(gridDim.x / a.kv_heads)) {
      most = 1;
      mine = count(b0, most, parts);
      end = sum_up_to(mine);
    }
    const int all = __builtin_amdgcn_readlane(end, 63);
    if (w < all) {
      const int who = (int)__builtin_ctzll(__ballot(end > w));
      const auto of = [&](int x) { return __builtin_amdgcn_readlane(x, who); };
      s = {of(s.q0), of(s.nq), of(s.k0), of(s.nk)};
      const int at = w - (of(end) - of(mine)), n = of(parts);
      return {b0 + who, at / n, at % n, most};
    }
    w -= all;
  }
  return {-1, 0, 0, 0};
}

// The number of a row's parts that a thread joins at a time: their loads are in flight together (2048 tokens: 9.4 us;
// 8 at a time 9.9, 16 11.0).
constexpr int kJoin = 4;

template <int D, bool F32, int WAVES>
__global__ __launch_bounds__(64 * WAVES, F32 || D == 128 || WAVES == 8 ? 2 : 3) void attn_few_kernel(AttnArgs a) {
  constexpr int NCT = D / 16, VE = F32 ? 4 : D / 16, NB = D / (16 * VE), NK = F32 ? D / 16 : D / 32;
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  typedef typename std::conditional<!F32 && D == 64, u32x2, u32x4>::type VRaw;
  __shared__ float so[WAVES][16][D + 4];
  __shared__ float2 sml[WAVES][16];
  __shared__ bool last;
  const int groups = (a.max_q * a.group + 15) / 16, h = blockIdx.x % a.kv_heads;
  AttnSeq sq;
  const Piece piece = piece_of(a, (int)(blockIdx.x / a.kv_heads), groups, sq);
  const int b = piece.b, group = piece.group, split = piece.split;
  if (b < 0) return;
  const int rows = sq.nq * a.group, r0 = group * 16, r1 = min(r0 + 16, rows);
  if (r0 >= rows) return;
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6), col = lane & 15, quad = lane >> 4;
  const int r = min(r0 + col, r1 - 1);
  const int lim = attn_limit(a, sq, r / a.group);
  const int lim_lo = attn_limit(a, sq, r0 / a.group), lim_hi = attn_limit(a, sq, (r1 - 1) / a.group);
  int parts, from, to;
  if (!attn_part(a, lim_hi, split, piece.most, parts, from, to)) return;

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
  u32x4 k[2][NK];
  VRaw v[2][4][NB];
  const auto load_k = [&](int j) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      const IO* p = kh + (int64_t)min(j + 16 * t + col, to - 1) * a.k.st;
#pragma unroll
      for (int s = 0; s < NK; ++s) k[t][s] = load_raw<16>(p + (F32 ? 16 * s + 4 * quad : 32 * s + 8 * quad));
    }
  };
  const auto load_v = [&](int j) {
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const IO* p = vh + (int64_t)min(j + 16 * t + 4 * quad + i, to - 1) * a.v.st + VE * col;
#pragma unroll
        for (int n = 0; n < NB; ++n) v[t][i][n] = load_raw<sizeof(VRaw)>(p + 16 * VE * n);
      }
  };
  // In bf16 K of the next step is on its way while this one's weights and outputs are worked out, and its V
  // while the next one's scores are: that needs the registers of two waves of a SIMD (8 ragged sequences of up
  // to 32768 tokens, 32 heads of 128 on 8: 81 us, three waves without it 85). After the last step the last key
  // is read again. In fp32, whose steps are twice as large, it does not pay (65536 tokens: 101 us, without 100).
  if (!F32 && from + 32 * wave < to) {
    load_k(from + 32 * wave);
    load_v(from + 32 * wave);
  }
  for (int j = from + 32 * wave; j < to; j += 32 * WAVES) {
    if constexpr (F32) {
      load_k(j);
      load_v(j);
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
    if constexpr (!F32) load_k(j + 32 * WAVES);
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
    float p[2][4];
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        p[t][i] = exp2_fast(s4[t][i] * a.scale - m_run);  // the product rounded like m, or they differ by up to half a step of it
        l_run += p[t][i];
      }
    if (strange) {  // values that are not finite become zero
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (j + 16 * t + 4 * quad + i < lim_lo) continue;
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < VE; ++e)
              if (not_finite(value_of<F32>(v[t][i][n], e))) v[t][i][n][F32 ? e : e / 2] &= F32 ? 0u : e % 2 ? 0xFFFFu : 0xFFFF0000u;
        }
    }
    if constexpr (F32) {
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int n = 0; n < NB; ++n)
#pragma unroll
            for (int e = 0; e < VE; ++e)
              o[VE * n + e] = __builtin_amdgcn_mfma_f32_16x16x4f32(value_of<F32>(v[t][i][n], e), p[t][i], o[VE * n + e], 0, 0, 0);
    } else {
      u32x4 hi, lo;  // the weights, and what their rounding to bf16 left of them
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float x = p[k / 2][k % 2 * 2], y = p[k / 2][k % 2 * 2 + 1];
        const uint32_t w = bf16_pair(x, y);
        hi[k] = w;
        lo[k] = bf16_pair(x - bf16_lo(w), y - bf16_hi(w));
      }
#pragma unroll
      for (int e = 0; e < VE; ++e) {
        u32x4 x;
#pragma unroll
        for (int k = 0; k < 4; ++k)  // channel e of two keys
          x[k] = __builtin_amdgcn_perm(v[k / 2][k % 2 * 2 + 1][0][e / 2], v[k / 2][k % 2 * 2][0][e / 2], e % 2 ? 0x07060302u : 0x05040100u);
        o[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, lo), o[e], 0, 0, 0);
        o[e] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8, x), __builtin_bit_cast(bf16x8, hi), o[e], 0, 0, 0);
      }
    }
    if constexpr (!F32) load_v(j + 32 * WAVES);
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
  if (WAVES > 4 && tid >= 256) return;
  const int d0 = (tid & 15) * NCT;
  int rr = tid >> 4;
  bool mine = r0 + rr < r1;
  float m = kLowest, l = 0.0f, f[WAVES];
#pragma unroll
  for (int w = 0; w < WAVES; ++w) m = fmaxf(m, sml[w][rr].x);
#pragma unroll
  for (int w = 0; w < WAVES; ++w) {
    f[w] = exp2_fast(sml[w][rr].x - m);
    l += sml[w][rr].y * f[w];
  }
  f32x4 x[NCT / 4];
#pragma unroll
  for (int i = 0; i < NCT / 4; ++i) {
    x[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < WAVES; ++w) x[i] += *reinterpret_cast<const f32x4*>(&so[w][rr][d0 + 4 * i]) * f[w];
  }
  if (WAVES == 4 && parts > 1) {
    // The part that is done last joins them all, in their order, so the result does not
    // depend on which one that was. Partial results pass between XCDs, whose L2 caches are
    // not coherent: they are written and read past them.
    const int64_t all = (int64_t)a.kv_heads * a.q_tokens * a.group;
    int64_t at = ((int64_t)h * a.q_tokens + sq.q0) * a.group + r0 + rr;
    if (mine) {
#pragma unroll
      for (int i = 0; i < NCT / 4; ++i) {
        put_pair(a.part + (split * all + at) * D + d0 + 4 * i, make_float2(x[i].x, x[i].y));
        put_pair(a.part + (split * all + at) * D + d0 + 4 * i + 2, make_float2(x[i].z, x[i].w));
      }
      if ((tid & 15) == 0) put_pair(&a.part_ml[split * all + at].x, make_float2(m, l));
    }
    uint32_t* arrived = a.arrived + ((int64_t)b * a.kv_heads + h) * groups + group;
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // this thread's stores are done
    __syncthreads();
    if (tid == 0) last = atomicAdd(arrived, 1u) == (uint32_t)parts - 1u;
    __syncthreads();
    if (!last) return;
    if (tid == 0) *arrived = 0;
    // With fewer rows than 16 several sets of threads take every sets-th part each.
    const int live = r1 - r0, sets = live > 8 ? 1 : live > 4 ? 2 : live > 2 ? 4 : live > 1 ? 8 : 16, set = rr * sets / 16;
    rr -= set * (16 / sets);
    at += rr - (tid >> 4);
    mine = rr < live;
    if (!mine) at -= rr - (live - 1);  // a row that is there, its result unused
    m = kLowest;
    l = 0.0f;
#pragma unroll
    for (int i = 0; i < NCT / 4; ++i) x[i] = f32x4{0, 0, 0, 0};
    for (int s0 = set; s0 < parts; s0 += kJoin * sets) {
      float2 ml[kJoin], y[kJoin][NCT / 2];
#pragma unroll
      for (int k = 0; k < kJoin; ++k) {
        const int64_t s = min(s0 + k * sets, parts - 1);
        ml[k] = get_pair(&a.part_ml[s * all + at].x);
#pragma unroll
        for (int i = 0; i < NCT / 2; ++i) y[k][i] = get_pair(a.part + (s * all + at) * D + d0 + 2 * i);
      }
#pragma unroll
      for (int k = 0; k < kJoin; ++k) {
        if (s0 + k * sets >= parts) break;
        const float m_new = fmaxf(m, ml[k].x), fo = exp2_fast(m - m_new), fs = exp2_fast(ml[k].x - m_new);
        m = m_new;
        l = l * fo + ml[k].y * fs;
#pragma unroll
        for (int i = 0; i < NCT / 4; ++i)
          x[i] = x[i] * fo + f32x4{y[k][2 * i].x, y[k][2 * i].y, y[k][2 * i + 1].x, y[k][2 * i + 1].y} * fs;
      }
    }
    if (sets > 1) {  // the sets of a row, in their order
      float(*const sx)[D + 4] = so[0];
      float2* const sm = sml[0];
      const int n = tid >> 4;
#pragma unroll
      for (int i = 0; i < NCT / 4; ++i) *reinterpret_cast<f32x4*>(&sx[n][d0 + 4 * i]) = x[i];
      if ((tid & 15) == 0) sm[n] = make_float2(m, l);
      __syncthreads();
      if (set) return;
      for (int k = 1; k < sets; ++k) {
        const int from_n = rr + k * (16 / sets);
        const float2 ml = sm[from_n];
        const float m_new = fmaxf(m, ml.x), fo = exp2_fast(m - m_new), fs = exp2_fast(ml.x - m_new);
        m = m_new;
        l = l * fo + ml.y * fs;
#pragma unroll
        for (int i = 0; i < NCT / 4; ++i) x[i] = x[i] * fo + *reinterpret_cast<const f32x4*>(&sx[from_n][d0 + 4 * i]) * fs;
      }
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
hipError_t run(const AttnArgs& a, int waves, int64_t pieces, hipStream_t s) {
  const int64_t grid = pieces * a.kv_heads;
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  constexpr int WIDE = 8;
  if (waves == 4) attn_few_kernel<D, F32, 4><<<(unsigned)grid, 256, 0, s>>>(a);
  else attn_few_kernel<D, F32, WIDE><<<(unsigned)grid, 64 * WIDE, 0, s>>>(a);
  return hipGetLastError();
}

}  // namespace

hipError_t launch_attn_few(const AttnArgs& a, bool bf16, int waves, int64_t pieces, hipStream_t s) {
  if (a.dim == 64) return bf16 ? run<64, false>(a, waves, pieces, s) : run<64, true>(a, waves, pieces, s);
  return bf16 ? run<128, false>(a, waves, pieces, s) : run<128, true>(a, waves, pieces, s);
}

}  // namespace rc
