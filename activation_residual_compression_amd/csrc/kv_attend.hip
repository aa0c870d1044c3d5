// Attention over the 8-bit key/value cache.
//
// Number formats. An e4m3 code is exact in f16, so K and V enter the f16 matrix
// instructions as they are and their block scales (powers of two) act on the fp32
// results. A query row is scaled by a power of two so that its largest value lies
// in [2^14, 2^15): a bf16 query is then exact in f16 (values under 2^-29 of the
// row's largest lose bits), and an fp32 query is the sum of two f16 (22 bits).
// Probabilities are rounded to f16 (11 bits) before they meet V where the outputs are
// bf16 (8 bits), or are the sum of two f16 for fp32; the sum of a row takes them as they
// were. Scores, statistics and outputs are accumulated in fp32. Two f16 for bf16 outputs
// too was measured: image share 138 -> 193 us, video share 701 -> 1002, prompts 94 -> 126,
// for an error against 64 bits of 1.659e-3 instead of 1.671e-3 (relative, of the whole
// output; the rounding to bf16 alone is 1.659e-3): not taken.
//
// Softmax in base 2: with c = scale * log2(e) * (scale of the row and block),
// p = 2^(S c - m + kBias), m the running maximum of S c (in the kernel for many rows
// only followed when p no longer fits f16, so the accumulators are rescaled a few
// times in all and not at every block). kBias lifts small probabilities out of f16's
// subnormals; both cancel in out = O / l.
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
// a lane's results runs of 8 (few rows) or 16 (many) consecutive tokens.
#include <type_traits>

#include "kv_device.hpp"

namespace rc {
namespace {

constexpr float kBias = 7.0f, kMost = 0x1p15f;  // f16 holds 2^15
constexpr int kEvUp = 2, kEvDown = 8;
// Rows of a block of threads of the kernel for many rows.
template <int D, bool F32>
constexpr int many_rows() { return D == 128 && F32 ? 32 : 64; }

// The rows of a call: row r of key head h is query r / G, query head h * G + r % G.
struct Row {
  int query, head;
};
__device__ __forceinline__ Row row_of(const KvAttendArgs& a, int h, int r) {
  return {r / a.g.group, h * a.g.group + r % a.g.group};
}

// Power of two that brings a row's largest value into [2^14, 2^15), and the exponent of
// its inverse. Rows under 2^-113 (2^127 is the largest factor) stay below 2^14.
__device__ __forceinline__ float row_scale(float top, int& down) {
  const int ex = (int)(__float_as_uint(top) >> 23 & 255);  // biased; 0: zero or subnormal
  down = max(ex - 141, -127);
  return pow2f(-down);
}

// Factor of a row's scores in a block: scale * 2^e, e the sum of the row's exponent and of
// the block's (-167 to 158), so that no product on the way leaves fp32 where the factor is
// in it. Not zero, even where a row and a block of zeros and a small scale meet: a masked
// score is -inf and has to stay it. What is raised to 2^-126 belongs to scores under 2^-90,
// which leave p at 1 either way. Not infinite, so that scores of zero stay it too.
__device__ __forceinline__ float factor_of(float scale, int e) {
  return fminf(fmaxf(ldexpf(scale, e), 0x1p-126f), -kLowest);
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

// Blocks that the queries of a tile see.
__device__ __forceinline__ int tile_reach(const KvAttendArgs& a, int len, int tile) {
  return (kv_limit(a, len, min((tile + 1) * a.q_tile, a.queries) - 1) + 63) / 64;
}

// A list of blocks ends at its first entry that is negative or not below `end`, the blocks
// that its tile sees; of the entries before, those up to the last one below `reach`, the
// blocks that these rows see. Called by whole waves.
__device__ __forceinline__ int list_length(const int32_t* list, int keep, int end, int reach, int lane) {
  int n = 0;
  for (int i = 0; i < keep; i += 64) {
    const int j = i + lane < keep ? list[i + lane] : -1;
    const uint64_t stop = __ballot(j < 0 || j >= end);
    const uint64_t seen = __ballot(j < reach) & (stop ? (stop & -stop) - 1 : ~(uint64_t)0);
    if (seen) n = i + 64 - __builtin_clzll(seen);
    if (stop) break;
  }
  return n;
}

// Takes in probability e of 16 (in order): the sum, and when it closes a pair, f16
// (and for fp32 what that left). Pinned in place, or the compiler gathers the sums and
// conversions of all 16 behind the last exponential, which takes registers.
template <bool F32>
__device__ __forceinline__ void take_p(const float (&p)[16], int e, float& sum, u32x4 (&ph)[2], u32x4 (&pl)[2]) {
  sum += p[e];
  if (e % 2 == 0) return;
  const half2_t hi = {(_Float16)p[e - 1], (_Float16)p[e]};
  uint32_t w = __builtin_bit_cast(uint32_t, hi);
  if constexpr (F32) {
    const half2_t lo = {(_Float16)(p[e - 1] - (float)hi.x), (_Float16)(p[e] - (float)hi.y)};
    uint32_t v = __builtin_bit_cast(uint32_t, lo);
    asm volatile("" : "+v"(v));
    pl[e / 8][e % 8 / 2] = v;
  }
  asm volatile("" : "+v"(w), "+v"(sum));
  ph[e / 8][e % 8 / 2] = w;
}
__device__ __forceinline__ half8_t as_half8(u32x4 x) { return __builtin_bit_cast(half8_t, x); }

// What a row's outputs are multiplied by at the end, and its log-sum-exp. Only a sum of
// zero is a row that sees nothing: one that is NaN stays NaN.
__device__ __forceinline__ float inverse_of(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float lse_of(float m, float l) { return l == 0.0f ? -INFINITY : (m - kBias + log2f(l)) * kLn2; }

// The part of a group's n blocks that this block of threads reads; parts: of how many.
__device__ __forceinline__ bool part_of(const KvAttendArgs& a, int n, int split, int& parts, int& from, int& to) {
  parts = min(max((n + a.chunk - 1) / a.chunk, 1), a.splits);
  const int per = (n + parts - 1) / parts;
  from = split * per;
  to = min(from + per, n);
  return split < parts;
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

// The blocks that a wave reads, entries from, from + step, ... below to, one after the
// other, without a load in the way: the wave's 64 lanes hold the next 64 (index, pool
// block, scales), loaded at once, and hand them out one by one. Blocks that do not
// exist are skipped, and those of a list that these rows do not see (from `reach` on).
struct Walk {
  const KvGeom& g;
  const int32_t* list;
  int b, h, base, to, step, reach, lane;
  uint64_t left;  // entries of these 64 still to come
  int lane_block;
  uint32_t lane_what;  // index (16 bits), exponents + 64 of K's and V's scales (8 bits each)

  __device__ __forceinline__ Walk(const KvGeom& g, const int32_t* list, int b, int h, int from, int to, int step,
                                  int reach, int lane)
      : g(g), list(list), b(b), h(h), base(from - 64 * step), to(to), step(step), reach(reach), lane(lane), left(0) {}
  __device__ __forceinline__ void fill() {
    base += 64 * step;
    lane_block = -1;
    const int at = base + lane * step;
    if (at < to) {
      const int j = list ? list[at] : at;
      lane_what = (uint32_t)j;
      if (j < reach) lane_block = kv_block(g, b, j);
    }
    if (lane_block >= 0) {
      const int64_t row = kv_row(g, lane_block, h);
      lane_what |= (uint32_t)(scale_exponent(g.k_scale[row]) + 64) << 16 | (uint32_t)(scale_exponent(g.v_scale[row]) + 64) << 24;
    }
    left = __ballot(lane_block >= 0);
  }
  // Moves to the next block: its index (-1: none) and pool block; `at` is its lane.
  __device__ __forceinline__ int next(int& block, int& at) {
    while (left == 0) {
      if (base + 64 * step >= to) return -1;
      fill();
    }
    at = __builtin_ctzll(left);
    left &= left - 1;
    block = __builtin_amdgcn_readlane(lane_block, at);
    return __builtin_amdgcn_readlane((int)lane_what, at) & 0xFFFF;
  }
  // Exponents of the scales of the block that next() found, before the next call of it.
  __device__ __forceinline__ void scales(int at, int& ks, int& ev) const {
    const uint32_t what = (uint32_t)__builtin_amdgcn_readlane((int)lane_what, at);
    ks = (int)(what >> 16 & 255u) - 64;
    ev = (int)(what >> 24) - 64;
  }
};

// ------------------------------------------------------------------ few rows
// One block of threads: 16 rows of one key head, a part of the keys. Each of its
// four waves reads blocks of its own straight into registers (a block's K and V
// are 16 loads of 16 B a lane) and keeps its own running maximum and sum; the four
// are joined in LDS, and the parts of the keys by the one that is done last. HBM
// bound: every code is read once for 16 rows. Three waves a SIMD without a prefetch
// beat two with the next block's loads in flight on long sequences (716 us against
// 739 for 64 of 32768 tokens). Measured with one query of four heads to a key head, 8
// key heads of 128: 64 sequences of 32768 tokens 710 us (6.05 TB/s), 4 of 65536 97 us
// (5.5), 32 ragged ones of up to 8192 61 us (5.0, in one part: a block of threads on each CU,
// which holds three, and most end before the longest), in fp32 91. One token over 333, 24
// heads: 7.2 us, most of it the launch and the chain of reads that wait for one another:
// length, queries, table, scales, codes (with lists two more).
template <int D, bool F32>
__global__ __launch_bounds__(256, F32 ? 2 : 3) void kv_attend_few_kernel(KvAttendArgs a) {
  constexpr int ND = D / 16, NQ = D / 64;
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  __shared__ float so[4][16][D + 4];
  __shared__ float2 sml[4][16];
  __shared__ bool last;
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
    count = list_length(list, a.keep, tile_reach(a, len, tile), reach, lane);
  }
  int parts, from, to;
  if (!part_of(a, count, split, parts, from, to)) return;

  half8_t qh[NQ][2], ql[NQ][2];
  int eq;  // the row's scores are 2^eq times the products
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
    const float up = row_scale(top, eq);
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
  Walk walk(g, list, b, h, from + wave, to, 4, reach, lane);
  int block, slot;
  for (int j; (j = walk.next(block, slot)) >= 0;) {
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
    float factor;
    int ks, ev;
    walk.scales(slot, ks, ev);
    const float ck = factor_of(a.scale, eq + ks);
    const int delta = enter_block(ev_cur, ev, factor);

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
  const bool mine = r0 + rr < r1;
  float m = kLowest, l = 0.0f, f[4];
#pragma unroll
  for (int w = 0; w < 4; ++w) m = fmaxf(m, sml[w][rr].x);
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    f[w] = exp2_fast(sml[w][rr].x - m);
    l += sml[w][rr].y * f[w];
  }
  f32x4 x[ND / 4];
#pragma unroll
  for (int i = 0; i < ND / 4; ++i) {
    x[i] = f32x4{0, 0, 0, 0};
#pragma unroll
    for (int w = 0; w < 4; ++w) x[i] += *reinterpret_cast<const f32x4*>(&so[w][rr][d0 + 4 * i]) * f[w];
  }
  if (parts > 1) {
    // The part that is done last joins them all, in their order, so the result does not
    // depend on which one that was. Partial results pass between XCDs, whose L2 caches
    // are not coherent: they are written and read past them (put_pair, get_pair). A
    // fence instead would write back the whole L2 for every block of threads (measured:
    // 368 us for a call that takes 65).
    const int64_t all = (int64_t)g.batch * g.kv_heads * rows, at = ((int64_t)b * g.kv_heads + h) * rows + r0 + rr;
    if (mine) {
#pragma unroll
      for (int i = 0; i < ND / 4; ++i) {
        put_pair(a.part + (split * all + at) * D + d0 + 4 * i, make_float2(x[i].x, x[i].y));
        put_pair(a.part + (split * all + at) * D + d0 + 4 * i + 2, make_float2(x[i].z, x[i].w));
      }
      if ((tid & 15) == 0) put_pair(&a.part_ml[split * all + at].x, make_float2(m, l));
    }
    uint32_t* arrived = a.arrived + ((int64_t)b * g.kv_heads + h) * (gridDim.x / a.splits) + group;
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
    for (int i = 0; i < ND / 4; ++i) x[i] = f32x4{0, 0, 0, 0};
    for (int s = 0; s < parts; ++s) {
      const float2 ml = get_pair(&a.part_ml[s * all + at].x);
      float2 y[ND / 2];
#pragma unroll
      for (int i = 0; i < ND / 2; ++i) y[i] = get_pair(a.part + (s * all + at) * D + d0 + 2 * i);
      const float m_new = fmaxf(m, ml.x), fo = exp2_fast(m - m_new), fs = exp2_fast(ml.x - m_new);
      m = m_new;
      l = l * fo + ml.y * fs;
#pragma unroll
      for (int i = 0; i < ND / 4; ++i)
        x[i] = x[i] * fo + f32x4{y[2 * i].x, y[2 * i].y, y[2 * i + 1].x, y[2 * i + 1].y} * fs;
    }
  }
  if (!mine) return;
  const Row to_row = row_of(a, h, r0 + rr);
  const float inv = inverse_of(l);
  IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)to_row.query * a.out.st + to_row.head * a.out.sh + d0;
#pragma unroll
  for (int i = 0; i < ND / 4; ++i) {
    const f32x4 y = x[i] * inv;
    if constexpr (F32)
      *reinterpret_cast<f32x4*>(out + 4 * i) = y;
    else
      *reinterpret_cast<u32x2*>(out + 4 * i) = u32x2{bf16_pair(y.x, y.y), bf16_pair(y.z, y.w)};
  }
  if (a.lse && (tid & 15) == 0)
    a.lse[((int64_t)b * a.queries + to_row.query) * g.q_heads + to_row.head] = lse_of(m, l);
}

// ------------------------------------------------------------------ many rows
// Which part of the call a block of threads does. They go to the 8 XCDs in turn. With one
// sequence whose rows all see the same, each XCD gets an equal run of the heads' tiles, so
// that a head's K and V pass through one L2 (4444 queries over 17776 tokens, 30 heads of
// 64: 695 us, 732 in plain order; over 70 chosen blocks each 220 and 228). Otherwise tiles
// are in order of length, the longest first, over all heads: runs would leave XCDs with
// the long sequences' tiles alone (three ragged causal sequences: 195 us in runs, 115 so),
// and one head to one XCD gained nothing (two of 24 heads of 128: 139 us either way). Where
// heads times sequences and 8 share a factor this order too keeps a sequence to some XCDs
// (two sequences of four heads: each to four of them).
struct Place {
  int b, h, split, tile;
};
__device__ __forceinline__ Place place_of(const KvAttendArgs& a, uint32_t w, uint32_t grid, int row_tiles) {
  const uint32_t per = (uint32_t)(row_tiles * a.splits), heads = (uint32_t)a.g.kv_heads;
  uint32_t in_head, b, h;
  if (!a.causal && a.g.batch == 1) {
    const uint32_t xcd = w & 7u;
    w = xcd * (grid >> 3) + min(xcd, grid & 7u) + (w >> 3);
    in_head = w % per;
    h = w / per;
    b = 0;
  } else {
    const uint32_t all = heads * (uint32_t)a.g.batch;
    in_head = w / all;
    w %= all;
    h = w % heads;
    b = w / heads;
  }
  const int tile = (int)in_head / a.splits;
  return {(int)b, (int)h, (int)in_head % a.splits, a.causal ? row_tiles - 1 - tile : tile};
}

// One block of threads: 64 rows of one key head, a part of the keys; its four waves
// read blocks of their own straight into registers, as in the kernel for few rows, so
// the loop has no barrier and no LDS write, and the waves of a SIMD drift apart: one
// does its softmax while another feeds the matrix units. All rows' queries are in LDS,
// written once; an operand of K or V serves two groups of 32 rows (one for fp32 at 128
// channels, whose registers hold no more). The waves are joined in LDS at the end.
//
// Against 128 rows with K and V widened into LDS by all waves (two buffers, a barrier a
// block): video share 764 -> 695 us, its block-selected form 250 -> 220, ragged causal
// prompts 110 -> 95, image share 139 -> 139, in fp32 135 -> 141; there LDS writes cost
// as much as the conversions. Bound by the vector units next to the matrix units: of
// their cycles 63 % and 51 % at 128 channels, 88 % and 47 % at 64 (exponentials, sums and
// the conversions of K and V, of which 64 rows share one). Measured: 1152 queries over
// 4608 tokens, 2 x 24 heads of 128, 138 to 144 us on different cards (up to 940 TFLOP/s);
// 4444 over 17776, 30 heads of 64, 695 to 723 us (up to 870).
template <int D, bool F32>
__global__ __launch_bounds__(256, D == 128 && !F32 ? 2 : 3) void kv_attend_many_kernel(KvAttendArgs a) {
  constexpr int NK = D / 16, ND = D / 32, ROWS = many_rows<D, F32>(), U = ROWS / 32;
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  constexpr int QBYTES = (F32 ? 2 : 1) * NK * 2 * ROWS * 16, OBYTES = 2 * ROWS * (D + 4) * 4;
  __shared__ __align__(16) char shared[QBYTES > OBYTES ? QBYTES : OBYTES];
  __shared__ float2 sml[4][ROWS];
  typedef half8_t QFrag[2][ROWS];
  QFrag* sq = reinterpret_cast<QFrag*>(shared);  // [hi: NK, lo: NK][half][row]: 8 channels of a row
  const KvGeom& g = a.g;
  const int rows = a.queries * g.group;
  const int row_tiles = (rows + ROWS - 1) / ROWS;
  const Place place = place_of(a, blockIdx.x, gridDim.x, row_tiles);
  const int b = place.b, h = place.h, split = place.split, tile = place.tile;
  const int r0 = tile * ROWS;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 31, half = lane >> 5;
  const int len = kv_length(a, b);
  const int lim_lo = r0 + ROWS > rows ? 0 : kv_limit(a, len, r0 / g.group);
  const int lim_hi = kv_limit(a, len, (min(r0 + ROWS, rows) - 1) / g.group);
  const int32_t* list = nullptr;
  const int reach = (lim_hi + 63) / 64;  // no block from here on, whatever a list says
  int count = reach;
  if (a.blocks) {
    list = a.blocks + (((int64_t)b * g.kv_heads + h) * a.tiles + (r0 / g.group) / a.q_tile) * a.keep;
    count = list_length(list, a.keep, tile_reach(a, len, (r0 / g.group) / a.q_tile), reach, lane);
  }
  int parts, from, to;
  if (!part_of(a, count, split, parts, from, to)) return;

  // Queries into LDS: 4 threads a row, every fourth 8 channels each. Operand f = 2 i + m,
  // half hh has channels 16 (2 i + hh) + 8 m + 0..7: so that 16 consecutive codes of K in
  // a lane are the operands of two matrix instructions.
  {
    const int r = tid >> 2 & (ROWS - 1), part = tid & 3;  // with 32 rows, each twice over
    const Row me = row_of(a, h, min(r0 + r, rows - 1));
    const IO* q = (const IO*)a.q.data + b * a.q.sb + (int64_t)me.query * a.q.st + me.head * a.q.sh;
    float x[D / 32][8], top = 0.0f;
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      row8<IO>(q + 32 * s + 8 * part, x[s]);
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(x[s][i]));
    }
    top = group_max<4>(top);
    int down;
    const float up = row_scale(top, down);
#pragma unroll
    for (int s = 0; s < D / 32; ++s) {
      half8_t hi, lo;
#pragma unroll
      for (int i = 0; i < 8; ++i) x[s][i] *= up;
      to_half<F32>(x[s], hi, lo);
      // channels 32 s + 8 part: i = s, hh = part / 2, m = part % 2
      sq[2 * s + part % 2][part / 2][r] = hi;
      if constexpr (F32) sq[NK + 2 * s + part % 2][part / 2][r] = lo;
    }
    if (part == 0) sml[0][r].x = (float)down;
  }
  __syncthreads();
  float m_run[U], l_run[U];
  int eq[U], lim[U];  // a row's scores are 2^eq times the products
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = r0 + 32 * u + col;
    eq[u] = (int)sml[0][32 * u + col].x;
    lim[u] = r < rows ? kv_limit(a, len, row_of(a, h, r).query) : 0;
    m_run[u] = kLowest;
    l_run[u] = 0.0f;
  }
  f32x16 o[U][ND];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int d = 0; d < ND; ++d) o[u][d] = f32x16{};
  int ev_cur = 0;

  // Operand row -> token of a half block, so that result i of a lane is token 16 half + i.
  const int token = (col & 3) | (col >> 3 & 1) << 2 | (col >> 4 & 1) << 3 | (col >> 2 & 1) << 4;
  const uint32_t k_at = (uint32_t)(half * 64 + token) * 16u, v_at = (uint32_t)(half * D + col) * 16u;
  u32x4 kr[NK / 2], vr[ND];
  const auto load_k = [&](int block, int u) {  // a scalar base and the lane's offset
    const uint8_t* k = g.k + kv_row(g, block, h) * (64 * D) + u * (32 * 16);
#pragma unroll
    for (int i = 0; i < NK / 2; ++i) kr[i] = *reinterpret_cast<const u32x4*>(k + (k_at + (uint32_t)i * (2 * 64 * 16)));
  };
  const auto load_v = [&](int block, int u) {
    const uint8_t* v = g.v + kv_row(g, block, h) * (64 * D) + u * (2 * D * 16);
#pragma unroll
    for (int d = 0; d < ND; ++d) vr[d] = *reinterpret_cast<const u32x4*>(v + (v_at + (uint32_t)d * (32 * 16)));
  };

  Walk walk(g, list, b, h, from + wave, to, 4, reach, lane);
  int block, slot, j = walk.next(block, slot);
  if (j >= 0) load_k(block, 0);
  while (j >= 0) {
    float factor;
    int ks, ev;
    walk.scales(slot, ks, ev);
    const int delta = enter_block(ev_cur, ev, factor);
    const float back = pow2f(-delta);
    if (factor != 1.0f) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int i = 0; i < 16; ++i) o[u][d][i] *= factor;
    }
    int block_n = block;
    const int j_n = walk.next(block_n, slot);
#pragma unroll
    for (int hb = 0; hb < 2; ++hb) {  // half blocks of 32 tokens
      load_v(block, hb);
      // The products ahead of a wave in its softmax, so that the matrix units are fed first
      // (bf16: image share 144 -> 141 us, video share 712 -> 700; fp32: no gain).
      if constexpr (!F32) __builtin_amdgcn_s_setprio(1);
      f32x16 s[U] = {};
      constexpr int AHEAD = 1;
      half8_t qf[NK][U];
#pragma unroll
      for (int f = 0; f < AHEAD; ++f)
#pragma unroll
        for (int u = 0; u < U; ++u) qf[f][u] = sq[f][half][32 * u + col];
#pragma unroll
      for (int f = 0; f < NK; ++f) {
        if (f + AHEAD < NK) {
#pragma unroll
          for (int u = 0; u < U; ++u) qf[f + AHEAD][u] = sq[f + AHEAD][half][32 * u + col];
        }
        const half8_t kf = codes8(kr[f / 2][2 * (f % 2)], kr[f / 2][2 * (f % 2) + 1]);
#pragma unroll
        for (int u = 0; u < U; ++u) {
          s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qf[f][u], s[u], 0, 0, 0);
          if constexpr (F32)
            s[u] = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, sq[NK + f][half][32 * u + col], s[u], 0, 0, 0);
        }
        __builtin_amdgcn_sched_barrier(0);
      }
      // K of the next half block, or past the end this block's again (not used)
      load_k(hb == 0 ? block : block_n, 1 - hb);
      if (j * 64 + 32 * hb + 32 > lim_lo) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          // by bits, not by comparisons, whose 32 results at once would spill scalars
          const int left = min(max(lim[u] - j * 64 - 32 * hb - 16 * half, 0), 16);
          const uint32_t seen = (1u << left) - 1u;
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t on = (uint32_t)((int32_t)(seen << (31 - i)) >> 31);
            s[u][i] = __uint_as_float((__float_as_uint(s[u][i]) & on) | (0xFF800000u & ~on));
          }
        }
        if (j * 64 + 64 > len) {
#pragma unroll
          for (int d = 0; d < ND; ++d) vr[d] = keep_codes(vr[d], len - j * 64 - 32 * hb - 16 * half);
        }
      }
      if constexpr (!F32) __builtin_amdgcn_s_setprio(0);
      u32x4 ph[U][2], pl[U][2];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const float ck = factor_of(a.scale, eq[u] + ks);
        const auto weigh = [&](float& sum) {
          const float off = kBias + (float)delta - m_run[u];
          float p[16];
          sum = 0.0f;
#pragma unroll
          for (int i = 0; i < 16; i += 4) {  // four at a time, so that they take few registers
#pragma unroll
            for (int k = i; k < i + 4; ++k) p[k] = exp2_fast(fmaf(s[u][k], ck, off));
#pragma unroll
            for (int k = i; k < i + 4; ++k) take_p<F32>(p, k, sum, ph[u], pl[u]);
            __builtin_amdgcn_sched_barrier(0);
          }
        };
        float sum;
        weigh(sum);
        // Probabilities in terms of an m that a row has left far behind do not fit f16.
        // Their sum shows it (it is over kMost before any of them is over what f16 holds),
        // so no maximum is taken until then.
        if (__any(sum > kMost)) {
          float top = fmaxf(s[u][0], s[u][1]);
#pragma unroll
          for (int i = 2; i < 16; ++i) top = fmaxf(top, s[u][i]);
          const float m_new = fmaxf(m_run[u], max_halves(top) * ck), alpha = exp2_fast(m_run[u] - m_new);
          l_run[u] *= alpha;
          m_run[u] = m_new;
#pragma unroll
          for (int d = 0; d < ND; ++d)
#pragma unroll
            for (int i = 0; i < 16; ++i) o[u][d][i] *= alpha;
          weigh(sum);
        }
        l_run[u] = fmaf(sum, back, l_run[u]);
      }
      if constexpr (!F32) __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const half8_t vf = codes8(vr[d][2 * m], vr[d][2 * m + 1]);
#pragma unroll
          for (int u = 0; u < U; ++u) {
            o[u][d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, as_half8(ph[u][m]), o[u][d], 0, 0, 0);
            if constexpr (F32)
              o[u][d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, as_half8(pl[u][m]), o[u][d], 0, 0, 0);
          }
        }
    }
    j = j_n;
    block = block_n;
  }

  // join the waves: each scales to the common maximum of a row; 2 and 3 hand theirs to 0
  // and 1, and 1 to 0's place, so the order of the sums is fixed
  __syncthreads();  // the queries are read
  {
    // the thread's place again, from its number alone: kept through the loop it would spill
    int tid = threadIdx.x;
    asm volatile("" : "+v"(tid));
    const int wave = tid >> 6, col = tid & 31, half = tid >> 5 & 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      l_run[u] += __shfl_xor(l_run[u], 32);
      if (half == 0) sml[wave][32 * u + col] = make_float2(m_run[u], l_run[u]);
    }
    __syncthreads();
    const float unit = pow2f(ev_cur);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float m = kLowest;
#pragma unroll
      for (int w = 0; w < 4; ++w) m = fmaxf(m, sml[w][32 * u + col].x);
      const float f = exp2_fast(m_run[u] - m) * unit;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int i = 0; i < 16; ++i) o[u][d][i] *= f;
    }
    typedef float ORow[D + 4];
    ORow* so = reinterpret_cast<ORow*>(shared);  // [2][ROWS] rows of outputs
    const auto each = [&](int slab, auto&& what) {
#pragma unroll
      for (int u = 0; u < U; ++u)
#pragma unroll
        for (int d = 0; d < ND; ++d)
#pragma unroll
          for (int q = 0; q < 4; ++q) {
            f32x4* at = reinterpret_cast<f32x4*>(&so[slab * ROWS + 32 * u + col][32 * d + 8 * q + 4 * half]);
            what(at, f32x4{o[u][d][4 * q], o[u][d][4 * q + 1], o[u][d][4 * q + 2], o[u][d][4 * q + 3]});
          }
    };
    if (wave >= 2) each(wave - 2, [](f32x4* at, f32x4 x) { *at = x; });
    __syncthreads();
    if (wave < 2) each(wave, [](f32x4* at, f32x4 x) { *at += x; });
    __syncthreads();
    // 4 threads a row
    {
      const int r = tid >> 2, part = tid & 3;
      if (r >= ROWS || r0 + r >= rows) return;
      float m = kLowest, l = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) m = fmaxf(m, sml[w][r].x);
#pragma unroll
      for (int w = 0; w < 4; ++w) l += sml[w][r].y * exp2_fast(sml[w][r].x - m);
      const int64_t at = ((int64_t)b * g.kv_heads + h) * rows + r0 + r, all = (int64_t)g.batch * g.kv_heads * rows;
      if (a.splits > 1 && split == 0 && part == 0) a.part_n[at] = parts;
      const Row me = row_of(a, h, r0 + r);
      const float inv = parts > 1 ? 1.0f : inverse_of(l);
      IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)me.query * a.out.st + me.head * a.out.sh;
#pragma unroll
      for (int s = 0; s < D / 16; ++s) {
        const int d = 16 * s + 4 * part;
        const f32x4 x = (*reinterpret_cast<const f32x4*>(&so[r][d]) + *reinterpret_cast<const f32x4*>(&so[ROWS + r][d])) * inv;
        if (parts > 1)
          *reinterpret_cast<f32x4*>(a.part + (split * all + at) * D + d) = x;
        else if constexpr (F32)
          *reinterpret_cast<f32x4*>(out + d) = x;
        else
          *reinterpret_cast<u32x2*>(out + d) = u32x2{bf16_pair(x.x, x.y), bf16_pair(x.z, x.w)};
      }
      if (part == 0) {
        if (parts > 1)
          a.part_ml[split * all + at] = make_float2(m, l);
        else if (a.lse)
          a.lse[((int64_t)b * a.queries + me.query) * g.q_heads + me.head] =
              lse_of(m, l);
      }
    }
  }
}

// ------------------------------------------------------------------ joining splits
// D / 4 lanes a row: out = sum O_s 2^(m_s - m) / sum l_s 2^(m_s - m), parts in order. HBM
// (or last-level cache) bound: 133 thousand rows of 64 in two parts, 21 us.
template <int D, bool F32>
__global__ __launch_bounds__(256) void kv_attend_join_kernel(KvAttendArgs a) {
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  constexpr int LANES = D / 4;
  const KvGeom& g = a.g;
  const int64_t rows = (int64_t)a.queries * g.group, all = rows * g.kv_heads * g.batch;
  const int64_t at = (int64_t)blockIdx.x * (256 / LANES) + threadIdx.x / LANES;
  const int d0 = threadIdx.x % LANES * 4;
  if (at >= all) return;
  const int parts = a.part_n[at];
  if (parts == 1) return;
  float m = kLowest, l = 0.0f;
  f32x4 x = {0, 0, 0, 0};
  for (int s = 0; s < parts; ++s) m = fmaxf(m, a.part_ml[s * all + at].x);
#pragma unroll 4
  for (int s = 0; s < parts; ++s) {
    const float2 ml = a.part_ml[s * all + at];
    const f32x4 o = *reinterpret_cast<const f32x4*>(a.part + (s * all + at) * D + d0);
    const float f = exp2_fast(ml.x - m);
    l += ml.y * f;
    x += o * f;
  }
  const int r = (int)(at % rows), h = (int)(at / rows % g.kv_heads), b = (int)(at / rows / g.kv_heads);
  const Row me = row_of(a, h, r);
  x *= inverse_of(l);
  IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)me.query * a.out.st + me.head * a.out.sh + d0;
  if constexpr (F32)
    *reinterpret_cast<f32x4*>(out) = x;
  else
    *reinterpret_cast<u32x2*>(out) = u32x2{bf16_pair(x.x, x.y), bf16_pair(x.z, x.w)};
  if (a.lse && d0 == 0)
    a.lse[((int64_t)b * a.queries + me.query) * g.q_heads + me.head] = lse_of(m, l);
}

template <int D, bool F32>
hipError_t run(const KvAttendArgs& a, bool few, hipStream_t s) {
  const int64_t rows = (int64_t)a.queries * a.g.group;
  if (few) {
    const int64_t groups = a.blocks && a.q_tile == 1 ? (int64_t)a.queries * ((a.g.group + 15) / 16) : (rows + 15) / 16;
    const dim3 grid((unsigned)(a.splits * groups), (unsigned)a.g.kv_heads, (unsigned)a.g.batch);
    kv_attend_few_kernel<D, F32><<<grid, 256, 0, s>>>(a);
  } else {
    const int64_t grid = a.splits * ((rows + many_rows<D, F32>() - 1) / many_rows<D, F32>()) * a.g.kv_heads * a.g.batch;
    if (grid > INT32_MAX) return hipErrorInvalidValue;
    kv_attend_many_kernel<D, F32><<<(unsigned)grid, 256, 0, s>>>(a);
  }
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && a.splits > 1 && !few) {
    const int64_t per = 256 / (D / 4);
    kv_attend_join_kernel<D, F32><<<(unsigned)((rows * a.g.kv_heads * a.g.batch + per - 1) / per), 256, 0, s>>>(a);
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
