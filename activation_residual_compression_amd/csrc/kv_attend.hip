// Attention over the 8-bit key/value cache.
//
// Number formats. An e4m3 code is exact in f16, so K and V enter the f16 matrix
// instructions as they are and their block scales (powers of two) act on the fp32
// results. A query row is scaled by a power of two so that its largest value lies
// in [2^14, 2^15): a bf16 query is then exact in f16 (values under 2^-29 of the
// row's largest lose bits), and an fp32 query is the sum of two f16 (22 bits).
// Probabilities are rounded to f16 (11 bits; bf16 outputs keep 8), or are the sum
// of two f16 for fp32. Scores, statistics and outputs are accumulated in fp32.
//
// Softmax in base 2: with c = scale * log2(e) * (scale of the row and block),
// p = 2^(S c - m + kBias), m the running maximum of S c. kBias lifts small
// probabilities out of f16's subnormals; it cancels in out = O / l.
//
// V's exponent ev differs from block to block. The output accumulators hold units
// of 2^ev_cur: while ev is near ev_cur the difference goes into the exponent of p
// (and is taken back from the block's sum, once), else the accumulators are
// rescaled (exact). |ev - ev_cur| can be 84 at most, which fp32 holds.
//
// Both kernels compute S^T = K Q^T and O^T = V^T P^T: a lane then holds scores of
// one query only (its column), the softmax is in the lane, and the fp32 scores of
// S^T are, rounded to f16 and with no exchange between lanes, the B operand of the
// second product. For that, rows of the K operand are taken in an order that makes
// the 8 results of a lane 8 consecutive tokens.
#include <type_traits>

#include "kv_device.hpp"

namespace rc {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kBias = 8.0f;      // p <= 2^(8 + 2): f16 holds 2^15
constexpr int kEvUp = 2, kEvDown = 8;
constexpr float kLowest = -3.402823466e38f;

__device__ __forceinline__ float exp2_fast(float x) { return __builtin_amdgcn_exp2f(x); }

// The rows of a call: row r of key head h is query r / G, query head h * G + r % G.
struct Row {
  int query, head;
};
__device__ __forceinline__ Row row_of(const KvAttendArgs& a, int h, int r) {
  return {r / a.g.group, h * a.g.group + r % a.g.group};
}

// Power of two that brings a row's largest value into [2^14, 2^15), and its inverse.
__device__ __forceinline__ void row_scale(float top, float& up, float& down) {
  const int ex = (int)(__float_as_uint(top) >> 23 & 255);  // biased; 0: zero or subnormal
  const int e = min(max(141 - ex, -100), 100);
  up = pow2f(e);
  down = pow2f(-e);
}

// Before a block of exponent ev: what goes into the exponent of p, and the factor
// of the accumulators (1: nothing to do).
__device__ __forceinline__ int enter_block(int& ev_cur, int ev, float& factor) {
  int delta = ev - ev_cur;
  factor = 1.0f;
  if (delta > kEvUp || delta < -kEvDown) {
    factor = pow2f(-delta);
    ev_cur = ev;
    delta = 0;
  }
  return delta;
}

// The lane's 8 probabilities as f16, and for fp32 what that rounding left.
template <bool F32>
__device__ __forceinline__ void to_half(const float (&p)[8], half8_t& hi, half8_t& lo) {
#pragma unroll
  for (int i = 0; i < 8; ++i) hi[i] = (_Float16)p[i];
  if constexpr (F32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) lo[i] = (_Float16)(p[i] - (float)hi[i]);
  }
}

// Entries of a list of blocks before the first one that is negative or not below
// `reach`. Called by whole waves.
__device__ __forceinline__ int list_length(const int32_t* list, int keep, int reach, int lane) {
  for (int i = 0; i < keep; i += 64) {
    const int j = i + lane < keep ? list[i + lane] : -1;
    const uint64_t end = __ballot(j < 0 || j >= reach);
    if (end) return i + __builtin_ctzll(end);
  }
  return keep;
}

// Keeps the first n of the 16 codes of u (n <= 0: none), so that stale codes after
// a sequence's end never meet a probability of zero as a NaN.
__device__ __forceinline__ u32x4 keep_codes(u32x4 u, int n) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int left = n - 4 * i;
    const uint32_t mask = left >= 4 ? 0xFFFFFFFFu : left <= 0 ? 0u : (1u << (8 * left)) - 1u;
    u[i] &= mask;
  }
  return u;
}

// ------------------------------------------------------------------ few rows
// One block of threads: 16 rows of one key head, a part of the keys. Each of its
// four waves reads blocks of its own straight into registers (a block's K and V
// are 16 loads of 16 B a lane) and keeps its own running maximum and sum; the four
// are joined in LDS. HBM bound: every code is read once for 16 rows.
template <int D, bool F32>
__global__ __launch_bounds__(256, 2) void kv_attend_few_kernel(KvAttendArgs a) {
  constexpr int ND = D / 16, NQ = D / 64;
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  __shared__ float so[4][16][D + 4];
  __shared__ float2 sml[4][16];
  const KvGeom& g = a.g;
  // groups of 16 rows do not cross what shares a list of blocks: with q_tile 1 a query's rows (span)
  const int rows = a.queries * g.group, span = a.blocks && a.q_tile == 1 ? g.group : rows;
  const int per_span = (span + 15) / 16;
  const int b = blockIdx.z, h = blockIdx.y, split = blockIdx.x % a.splits, group = blockIdx.x / a.splits;
  const int r0 = group / per_span * span + group % per_span * 16, r1 = min(r0 + 16, (group / per_span + 1) * span);
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 15, quad = lane >> 4;
  const int r = r0 + col;
  const bool live = r < r1;
  const Row me = row_of(a, h, min(r, r1 - 1));
  const int len = kv_length(a, b);
  const int lim = live ? kv_limit(a, len, me.query) : 0;
  const int lim_lo = kv_limit(a, len, r0 / g.group);
  const int lim_hi = kv_limit(a, len, (r1 - 1) / g.group);
  const int32_t* list = nullptr;
  const int reach = (lim_hi + 63) / 64;  // no block from here on, whatever a list says
  int count = reach;
  if (a.blocks) {
    const int tile = (r0 / g.group) / a.q_tile;
    list = a.blocks + (((int64_t)b * g.kv_heads + h) * a.tiles + tile) * a.keep;
    count = list_length(list, a.keep, reach, lane);
  }
  const int per = (count + a.splits - 1) / a.splits;
  const int from = split * per, to = min(from + per, count);

  half8_t qh[NQ][2], ql[NQ][2];
  float cq;
  {
    float x[NQ][2][8], top = 0.0f;
#pragma unroll
    for (int s = 0; s < NQ; ++s)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        row8<IO>((const IO*)a.q.data + b * a.q.sb + (int64_t)me.query * a.q.st + me.head * a.q.sh + 64 * s +
                     16 * quad + 8 * m, x[s][m]);
#pragma unroll
        for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[s][m][i]));
      }
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    float up, down;
    row_scale(top, up, down);
    cq = down * (a.scale * kLog2e);
#pragma unroll
    for (int s = 0; s < NQ; ++s)
#pragma unroll
      for (int m = 0; m < 2; ++m) {
        float y[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) y[i] = x[s][m][i] * up;
        to_half<F32>(y, qh[s][m], ql[s][m]);
      }
  }

  f32x4 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = f32x4{0, 0, 0, 0};
  float m_run = kLowest, l_run = 0.0f;
  int ev_cur = 0;
  for (int it = from + wave; it < to; it += 4) {
    const int j = list ? list[it] : it;
    const int block = kv_block(g, b, j);
    if (block < 0) continue;
    const int64_t row = kv_row(g, block, h);
    const uint8_t* kb = g.k + row * (64 * D);
    const uint8_t* vb = g.v + row * (64 * D);
    u32x4 k[4][NQ], v[ND];
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int s = 0; s < NQ; ++s)
        k[t][s] = *reinterpret_cast<const u32x4*>(kb + ((4 * s + quad) * 64 + 16 * (col >> 2) + 4 * t + (col & 3)) * 16);
#pragma unroll
    for (int d = 0; d < ND; ++d) v[d] = *reinterpret_cast<const u32x4*>(vb + (quad * D + 16 * d + col) * 16);
    const float ck = cq * g.k_scale[row];
    float factor;
    const int delta = enter_block(ev_cur, scale_exponent(g.v_scale[row]), factor);

    f32x4 s4[4];
#pragma unroll
    for (int t = 0; t < 4; ++t) {
      s4[t] = f32x4{0, 0, 0, 0};
#pragma unroll
      for (int s = 0; s < NQ; ++s)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const half8_t kf = codes8(k[t][s][2 * m], k[t][s][2 * m + 1]);
          s4[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, qh[s][m], s4[t], 0, 0, 0);
          if constexpr (F32) s4[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(kf, ql[s][m], s4[t], 0, 0, 0);
        }
    }
    if (j * 64 + 64 > lim_lo || r1 - r0 < 16) {
      const int left = lim - j * 64 - 16 * quad;  // this lane's tokens are 16 quad + 4 t + i
#pragma unroll
      for (int t = 0; t < 4; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i)
          if (4 * t + i >= left) s4[t][i] = -INFINITY;
      if (j * 64 + 64 > len) {
#pragma unroll
        for (int d = 0; d < ND; ++d) v[d] = keep_codes(v[d], len - j * 64 - 16 * quad);
      }
    }
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 4; ++t)
#pragma unroll
      for (int i = 0; i < 4; ++i) top = fmaxf(top, s4[t][i]);
    top = fmaxf(top, __shfl_xor(top, 16));
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m_new = fmaxf(m_run, top * ck);
    if (__any(m_new > m_run) || factor != 1.0f) {
      const float alpha = exp2_fast(m_run - m_new);
      l_run *= alpha;
      const float f = alpha * factor;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 4; ++i) o[d][i] *= f;
      m_run = m_new;
    }
    const float off = kBias + (float)delta - m_run;
    float sum = 0.0f;
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_fast(fmaf(s4[2 * m + i / 4][i % 4], ck, off));
        sum += p[i];
      }
      half8_t ph, pl;
      to_half<F32>(p, ph, pl);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const half8_t vf = codes8(v[d][2 * m], v[d][2 * m + 1]);
        o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, ph, o[d], 0, 0, 0);
        if constexpr (F32) o[d] = __builtin_amdgcn_mfma_f32_16x16x32_f16(vf, pl, o[d], 0, 0, 0);
      }
    }
    l_run = fmaf(sum, pow2f(-delta), l_run);
  }
  l_run += __shfl_xor(l_run, 16);
  l_run += __shfl_xor(l_run, 32);
  const float unit = pow2f(ev_cur);
#pragma unroll
  for (int d = 0; d < ND; ++d)
    *reinterpret_cast<f32x4*>(&so[wave][col][16 * d + 4 * quad]) = o[d] * unit;
  if (quad == 0) sml[wave][col] = make_float2(m_run, l_run);
  __syncthreads();

  // join the waves: 16 threads a row, D / 16 values each
  const int rr = tid >> 4, d0 = (tid & 15) * ND;
  if (r0 + rr >= r1) return;
  float m = kLowest, l = 0.0f, f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) m = fmaxf(m, sml[w][rr].x);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = exp2_fast(sml[w][rr].x - m);
    l += sml[w][rr].y * f[w];
  }
  float x[ND];
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    x[i] = 0.0f;
#pragma unroll
    for (int w = 0; w < 4; ++w) x[i] += so[w][rr][d0 + i] * f[w];
  }
  if (a.splits > 1) {
    const int64_t at = ((int64_t)split * g.batch + b) * g.kv_heads * rows + (int64_t)h * rows + r0 + rr;
#pragma unroll
    for (int i = 0; i < ND; ++i) a.part[at * D + d0 + i] = x[i];
    if ((tid & 15) == 0) a.part_ml[at] = make_float2(m, l);
    return;
  }
  const Row to_row = row_of(a, h, r0 + rr);
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)to_row.query * a.out.st + to_row.head * a.out.sh + d0;
#pragma unroll
  for (int i = 0; i < ND; ++i) {
    if constexpr (F32) out[i] = x[i] * inv;
    else out[i] = (uint16_t)bf16_rne(x[i] * inv);
  }
  if (a.lse && (tid & 15) == 0)
    a.lse[((int64_t)b * a.queries + to_row.query) * g.q_heads + to_row.head] =
        l > 0.0f ? (m - kBias + log2f(l)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------------ many rows
// One block of threads: 128 rows of one key head (32 a wave). K and V of a block
// are widened to f16 once, on their way into LDS (two buffers: the next block's
// loads are in flight while this one is computed), in the order of the operands,
// so that every LDS read is one run of 64 lanes x 16 B.
template <int D, bool F32>
__global__ __launch_bounds__(256, 2) void kv_attend_many_kernel(KvAttendArgs a) {
  constexpr int NK = D / 16, ND = D / 32, UNITS = 64 * D / 16 / 256;
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  __shared__ half8_t sk[2][D / 8][64];  // [channel / 8][operand row]
  __shared__ half8_t sv[2][8][D];       // [token / 8][channel]
  const KvGeom& g = a.g;
  const int b = blockIdx.z, h = blockIdx.y;
  const int rows = a.queries * g.group;
  const int row_tiles = (rows + 127) / 128;
  const int split = blockIdx.x / row_tiles;
  const int tile = a.causal ? row_tiles - 1 - blockIdx.x % row_tiles : blockIdx.x % row_tiles;  // long rows first
  const int r0 = tile * 128;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 31, half = lane >> 5;
  const int r = r0 + wave * 32 + col;
  const bool live = r < rows;
  const Row me = row_of(a, h, min(r, rows - 1));
  const int len = kv_length(a, b);
  const int lim = live ? kv_limit(a, len, me.query) : 0;
  const int lim_lo = kv_limit(a, len, r0 / g.group);
  const int lim_hi = kv_limit(a, len, (min(r0 + 128, rows) - 1) / g.group);
  const int32_t* list = nullptr;
  const int reach = (lim_hi + 63) / 64;  // no block from here on, whatever a list says
  int count = reach;
  if (a.blocks) {
    list = a.blocks + (((int64_t)b * g.kv_heads + h) * a.tiles + (r0 / g.group) / a.q_tile) * a.keep;
    count = list_length(list, a.keep, reach, lane);
  }
  const int per = (count + a.splits - 1) / a.splits;
  const int from = split * per, to = min(from + per, count);

  half8_t qh[NK], ql[NK];
  float cq;
  {
    float top = 0.0f;
    const IO* q = (const IO*)a.q.data + b * a.q.sb + (int64_t)me.query * a.q.st + me.head * a.q.sh + 8 * half;
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      float x[8];
      row8<IO>(q + 16 * s, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[i]));
    }
    top = fmaxf(top, __shfl_xor(top, 32));
    float up, down;
    row_scale(top, up, down);
    cq = down * (a.scale * kLog2e);
#pragma unroll
    for (int s = 0; s < NK; ++s) {
      float x[8];
      row8<IO>(q + 16 * s, x);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] *= up;
      to_half<F32>(x, qh[s], ql[s]);
    }
  }

  // the next block that exists, at or after it; -1 at the end
  const auto next = [&](int& it, int& block) {
    for (; it < to; ++it) {
      const int j = list ? list[it] : it;
      block = kv_block(g, b, j);
      if (block >= 0) return j;
    }
    return -1;
  };
  u32x4 kr[UNITS], vr[UNITS];
  const auto load = [&](int block) {
    const int64_t row = kv_row(g, block, h);
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int unit = tid + 256 * u, p = unit & 63;
      const int t = (p & ~12) | (p & 4) << 1 | (p & 8) >> 1;  // operand row -> token: bits 2 and 3 change places
      kr[u] = *reinterpret_cast<const u32x4*>(g.k + row * (64 * D) + ((unit & ~63) | t) * 16);
      vr[u] = *reinterpret_cast<const u32x4*>(g.v + row * (64 * D) + unit * 16);
    }
  };
  const auto stage = [&](int buf, int j) {
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      const int unit = tid + 256 * u;
      sk[buf][2 * (unit >> 6)][unit & 63] = codes8(kr[u][0], kr[u][1]);
      sk[buf][2 * (unit >> 6) + 1][unit & 63] = codes8(kr[u][2], kr[u][3]);
      u32x4 w = vr[u];
      if (j * 64 + 64 > len) w = keep_codes(w, len - j * 64 - 16 * (unit / D));
      sv[buf][2 * (unit / D)][unit % D] = codes8(w[0], w[1]);
      sv[buf][2 * (unit / D) + 1][unit % D] = codes8(w[2], w[3]);
    }
  };

  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = f32x16{};
  float m_run = kLowest, l_run = 0.0f;
  int ev_cur = 0, it = from, block = -1, buf = 0;
  int j = next(it, block);
  if (j >= 0) {
    load(block);
    stage(0, j);
  }
  while (j >= 0) {
    const int64_t row = kv_row(g, block, h);
    const float ck = cq * g.k_scale[row];
    float factor;
    const int delta = enter_block(ev_cur, scale_exponent(g.v_scale[row]), factor);
    int block_n = -1;
    ++it;
    const int j_n = next(it, block_n);
    if (j_n >= 0) load(block_n);
    __syncthreads();

    f32x16 s16[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      s16[t] = f32x16{};
#pragma unroll
      for (int s = 0; s < NK; ++s) {
        const half8_t kf = sk[buf][2 * s + half][32 * t + col];
        s16[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qh[s], s16[t], 0, 0, 0);
        if constexpr (F32) s16[t] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, ql[s], s16[t], 0, 0, 0);
      }
    }
    if (j * 64 + 64 > lim_lo || r0 + 128 > rows) {
      const int left = lim - j * 64 - 8 * half;  // result i of tile t is token 32 t + 16 (i / 8) + 8 half + i % 8
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < 16; ++i)
          if (32 * t + 16 * (i / 8) + i % 8 >= left) s16[t][i] = -INFINITY;
    }
    float top = -INFINITY;
#pragma unroll
    for (int t = 0; t < 2; ++t)
#pragma unroll
      for (int i = 0; i < 16; ++i) top = fmaxf(top, s16[t][i]);
    top = fmaxf(top, __shfl_xor(top, 32));
    const float m_new = fmaxf(m_run, top * ck);
    if (__any(m_new > m_run) || factor != 1.0f) {
      const float alpha = exp2_fast(m_run - m_new);
      l_run *= alpha;
      const float f = alpha * factor;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[d][i] *= f;
      m_run = m_new;
    }
    const float off = kBias + (float)delta - m_run;
    float sum = 0.0f;
#pragma unroll
    for (int s = 0; s < 4; ++s) {
      float p[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        p[i] = exp2_fast(fmaf(s16[s / 2][8 * (s % 2) + i], ck, off));
        sum += p[i];
      }
      half8_t ph, pl;
      to_half<F32>(p, ph, pl);
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const half8_t vf = sv[buf][2 * s + half][32 * d + col];
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, ph, o[d], 0, 0, 0);
        if constexpr (F32) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, pl, o[d], 0, 0, 0);
      }
    }
    l_run = fmaf(sum, pow2f(-delta), l_run);
    // the other buffer was last read before this iteration's barrier
    if (j_n >= 0) stage(buf ^ 1, j_n);
    buf ^= 1;
    j = j_n;
    block = block_n;
  }
  l_run += __shfl_xor(l_run, 32);
  if (!live) return;
  const float unit = pow2f(ev_cur);
  if (a.splits > 1) {
    const int64_t at = ((int64_t)split * g.batch + b) * g.kv_heads * rows + (int64_t)h * rows + r;
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int q = 0; q < 4; ++q)
        *reinterpret_cast<f32x4*>(a.part + at * D + 32 * d + 8 * q + 4 * half) =
            f32x4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]} * unit;
    if (half == 0) a.part_ml[at] = make_float2(m_run, l_run);
    return;
  }
  const float inv = l_run > 0.0f ? unit / l_run : 0.0f;
  IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)me.query * a.out.st + me.head * a.out.sh + 4 * half;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int q = 0; q < 4; ++q) {
      const f32x4 x = f32x4{o[d][4 * q], o[d][4 * q + 1], o[d][4 * q + 2], o[d][4 * q + 3]} * inv;
      if constexpr (F32)
        *reinterpret_cast<f32x4*>(out + 32 * d + 8 * q) = x;
      else
        *reinterpret_cast<u32x2*>(out + 32 * d + 8 * q) =
            u32x2{bf16_rne(x.x) | bf16_rne(x.y) << 16, bf16_rne(x.z) | bf16_rne(x.w) << 16};
    }
  if (a.lse && half == 0)
    a.lse[((int64_t)b * a.queries + me.query) * g.q_heads + me.head] =
        l_run > 0.0f ? (m_run - kBias + log2f(l_run)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------------ joining splits
// One wave a row: out = sum O_s 2^(m_s - m) / sum l_s 2^(m_s - m).
template <int D, bool F32>
__global__ __launch_bounds__(256) void kv_attend_join_kernel(KvAttendArgs a) {
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  constexpr int W = D / 64;
  const KvGeom& g = a.g;
  const int64_t rows = (int64_t)a.queries * g.group, all = rows * g.kv_heads * g.batch;
  const int64_t at = (int64_t)blockIdx.x * 4 + (threadIdx.x >> 6);
  const int lane = threadIdx.x & 63;
  if (at >= all) return;
  float m = kLowest, l = 0.0f, x[W];
#pragma unroll
  for (int i = 0; i < W; ++i) x[i] = 0.0f;
  for (int s = 0; s < a.splits; ++s) m = fmaxf(m, a.part_ml[s * all + at].x);
  for (int s = 0; s < a.splits; ++s) {
    const float2 ml = a.part_ml[s * all + at];
    const float f = exp2_fast(ml.x - m);
    l += ml.y * f;
#pragma unroll
    for (int i = 0; i < W; ++i) x[i] += a.part[(s * all + at) * D + lane * W + i] * f;
  }
  const int r = (int)(at % rows), h = (int)(at / rows % g.kv_heads), b = (int)(at / rows / g.kv_heads);
  const Row me = row_of(a, h, r);
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)me.query * a.out.st + me.head * a.out.sh + lane * W;
#pragma unroll
  for (int i = 0; i < W; ++i) {
    if constexpr (F32) out[i] = x[i] * inv;
    else out[i] = (uint16_t)bf16_rne(x[i] * inv);
  }
  if (a.lse && lane == 0)
    a.lse[((int64_t)b * a.queries + me.query) * g.q_heads + me.head] =
        l > 0.0f ? (m - kBias + log2f(l)) * kLn2 : -INFINITY;
}

template <int D, bool F32>
hipError_t run(const KvAttendArgs& a, bool few, hipStream_t s) {
  const int64_t rows = (int64_t)a.queries * a.g.group;
  if (few) {
    const int64_t groups = a.blocks && a.q_tile == 1 ? (int64_t)a.queries * ((a.g.group + 15) / 16) : (rows + 15) / 16;
    const dim3 grid((unsigned)(a.splits * groups), (unsigned)a.g.kv_heads, (unsigned)a.g.batch);
    kv_attend_few_kernel<D, F32><<<grid, 256, 0, s>>>(a);
  } else {
    const dim3 grid((unsigned)(a.splits * ((rows + 127) / 128)), (unsigned)a.g.kv_heads, (unsigned)a.g.batch);
    kv_attend_many_kernel<D, F32><<<grid, 256, 0, s>>>(a);
  }
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && a.splits > 1) {
    kv_attend_join_kernel<D, F32><<<(unsigned)((rows * a.g.kv_heads * a.g.batch + 3) / 4), 256, 0, s>>>(a);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace

hipError_t launch_kv_attend(const KvAttendArgs& a, bool few, bool bf16, hipStream_t s) {
  if (a.g.dim == 64) return bf16 ? run<64, false>(a, few, s) : run<64, true>(a, few, s);
  return bf16 ? run<128, false>(a, few, s) : run<128, true>(a, few, s);
}

}  // namespace rc
