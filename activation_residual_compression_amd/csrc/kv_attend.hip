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
// the 8 results of a lane 8 consecutive tokens.
#include <type_traits>

#include "kv_device.hpp"

namespace rc {
namespace {

constexpr float kLog2e = 1.44269504088896340736f, kLn2 = 0.69314718055994530942f;
constexpr float kBias = 7.0f, kMost = 0x1p15f;  // f16 holds 2^15
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

// Takes in probability e of 16 (in order): the sum, and when it closes a pair, f16
// (and for fp32 what that left). Pinned in place: see the step of the many-row kernel.
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

// Two floats written to, read from, memory that every XCD sees.
__device__ __forceinline__ void put_pair(float* p, float2 x) {
  const uint64_t u = (uint64_t)__float_as_uint(x.y) << 32 | __float_as_uint(x.x);
  __hip_atomic_store(reinterpret_cast<uint64_t*>(p), u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float2 get_pair(const float* p) {
  const uint64_t u = __hip_atomic_load(reinterpret_cast<const uint64_t*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  return make_float2(__uint_as_float((uint32_t)u), __uint_as_float((uint32_t)(u >> 32)));
}

// The blocks that a wave reads, entries from, from + step, ... below to, one after the
// other, without a load in the way: the wave's 64 lanes hold the next 64 (index, pool
// block, scales), loaded at once, and hand them out one by one. Blocks that do not
// exist are skipped.
struct Walk {
  const KvGeom& g;
  const int32_t* list;
  int b, h, base, to, step, lane;
  uint64_t left;  // entries of these 64 still to come
  int lane_j, lane_block, lane_e;  // lane_e: the exponents of K's and V's scales, 16 bits each

  __device__ __forceinline__ Walk(const KvGeom& g, const int32_t* list, int b, int h, int from, int to, int step,
                                  int lane)
      : g(g), list(list), b(b), h(h), base(from - 64 * step), to(to), step(step), lane(lane), left(0) {}
  __device__ __forceinline__ void fill() {
    base += 64 * step;
    lane_block = -1;
    const int at = base + lane * step;
    if (at < to) {
      lane_j = list ? list[at] : at;
      lane_block = kv_block(g, b, lane_j);
    }
    if (lane_block >= 0) {
      const int64_t row = kv_row(g, lane_block, h);
      lane_e = scale_exponent(g.k_scale[row]) << 16 | (scale_exponent(g.v_scale[row]) & 0xFFFF);
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
    return __builtin_amdgcn_readlane(lane_j, at);
  }
  // Exponents of the scales of the block that next() found, before the next call of it.
  __device__ __forceinline__ void scales(int at, float& ks, int& ev) const {
    const int e = __builtin_amdgcn_readlane(lane_e, at);
    ks = pow2f(e >> 16);
    ev = (int16_t)e;
  }
  __device__ __forceinline__ int next(int& block, float& ks, int& ev) {
    int at;
    const int j = next(block, at);
    if (j >= 0) scales(at, ks, ev);
    return j;
  }
};

// ------------------------------------------------------------------ few rows
// One block of threads: 16 rows of one key head, a part of the keys. Each of its
// four waves reads blocks of its own straight into registers (a block's K and V
// are 16 loads of 16 B a lane) and keeps its own running maximum and sum; the four
// are joined in LDS, and the parts of the keys by the one that is done last. HBM bound: every code is read once for 16 rows.
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
    count = list_length(list, a.keep, reach, lane);
  }
  int parts, from, to;
  if (!part_of(a, count, split, parts, from, to)) return;

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
  Walk walk(g, list, b, h, from + wave, to, 4, lane);
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
    float ks, factor;
    int ev;
    walk.scales(slot, ks, ev);
    const float ck = cq * ks;
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
  const float inv = l > 0.0f ? 1.0f / l : 0.0f;
  IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)to_row.query * a.out.st + to_row.head * a.out.sh + d0;
#pragma unroll
  for (int i = 0; i < ND / 4; ++i) {
    const f32x4 y = x[i] * inv;
    if constexpr (F32)
      *reinterpret_cast<f32x4*>(out + 4 * i) = y;
    else
      *reinterpret_cast<u32x2*>(out + 4 * i) = u32x2{bf16_rne(y.x) | bf16_rne(y.y) << 16, bf16_rne(y.z) | bf16_rne(y.w) << 16};
  }
  if (a.lse && (tid & 15) == 0)
    a.lse[((int64_t)b * a.queries + to_row.query) * g.q_heads + to_row.head] =
        l > 0.0f ? (m - kBias + log2f(l)) * kLn2 : -INFINITY;
}

// ------------------------------------------------------------------ many rows
// Which part of the call a block of threads does. They go to the 8 XCDs in turn, so
// where the load of the XCDs stays even, a key head's row tiles are given to one XCD,
// whose L2 then holds its K and V: with a multiple of 8 key heads, head h to XCD h % 8
// (every XCD gets the same share of every sequence, however long); with one sequence
// whose rows all see the same, equal runs of the heads' tiles. Otherwise the tiles are
// in order of length, the longest first, over all heads. Measured on 1152 queries over
// 4608 tokens (2 x 24 heads of 128): 140 us, against 147 in plain order; the runs on
// three ragged causal sequences of 4 key heads: 195 us against 115 in plain order.
struct Place {
  int b, h, split, tile;
};
__device__ __forceinline__ Place place_of(const KvAttendArgs& a, uint32_t w, uint32_t grid, int row_tiles) {
  const uint32_t per = (uint32_t)(row_tiles * a.splits), heads = (uint32_t)a.g.kv_heads;
  uint32_t in_head, b, h;
  if (heads % 8 == 0) {
    const uint32_t xcd = w & 7u;
    w >>= 3;
    in_head = w % per;
    w /= per;
    h = w % (heads / 8) * 8 + xcd;
    b = w / (heads / 8);
  } else if (!a.causal && a.g.batch == 1) {
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

// The larger of a lane's value and that of the lane 32 away.
__device__ __forceinline__ float max_halves(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}

// One block of threads: 128 rows of one key head (32 a wave). K and V of a block
// are widened to f16 once, on their way into LDS, in the order of the operands, so
// that every LDS read is one run of 64 lanes x 16 B.
//
// The matrix units and the exponentials take about as long as each other, so a wave
// works on three half blocks (32 tokens) at once: the second product of half x - 1,
// the softmax of half x and the first product of half x + 1 do not depend on each
// other and are interleaved. K is therefore one block ahead of V in LDS (two buffers
// of each, one barrier a block), and the global loads are one block ahead of that.
// Waves of a SIMD: what the registers allow (D = 64 in 2 instead of 3: 830 us for the
// video share instead of 780; fp32 at D = 128 in 2 would spill).
template <int D, bool F32>
__global__ __launch_bounds__(256, D == 128 ? (F32 ? 1 : 2) : (F32 ? 2 : 3)) void kv_attend_many_kernel(KvAttendArgs a) {
  constexpr int NK = D / 16, ND = D / 32, UNITS = 64 * D / 16 / 256;
  typedef typename std::conditional<F32, float, uint16_t>::type IO;
  __shared__ half8_t sk[2][D / 8][64];  // [channel / 8][operand row]
  __shared__ half8_t sv[2][8][D];       // [token / 8][channel]
  const KvGeom& g = a.g;
  const int rows = a.queries * g.group;
  const int row_tiles = (rows + 127) / 128;
  const Place place = place_of(a, blockIdx.x, gridDim.x, row_tiles);
  const int b = place.b, h = place.h, split = place.split, tile = place.tile;
  const int r0 = tile * 128;
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6, col = lane & 31, half = lane >> 5;
  const int r = r0 + wave * 32 + col;
  const bool live = r < rows;
  const Row me = row_of(a, h, min(r, rows - 1));
  const int len = kv_length(a, b);
  const int lim = live ? kv_limit(a, len, me.query) : 0;
  const int lim_lo = r0 + 128 > rows ? 0 : kv_limit(a, len, r0 / g.group);
  const int lim_hi = kv_limit(a, len, (min(r0 + 128, rows) - 1) / g.group);
  const int32_t* list = nullptr;
  const int reach = (lim_hi + 63) / 64;  // no block from here on, whatever a list says
  int count = reach;
  if (a.blocks) {
    list = a.blocks + (((int64_t)b * g.kv_heads + h) * a.tiles + (r0 / g.group) / a.q_tile) * a.keep;
    count = list_length(list, a.keep, reach, lane);
  }
  int parts, from, to;
  if (!part_of(a, count, split, parts, from, to)) return;

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
    top = max_halves(top);
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

  u32x4 kr[UNITS], vr[UNITS];
  const auto load_k = [&](int block, int u) {
    const int unit = tid + 256 * u, p = unit & 63;
    const int t = (p & ~12) | (p & 4) << 1 | (p & 8) >> 1;  // operand row -> token: bits 2 and 3 change places
    kr[u] = *reinterpret_cast<const u32x4*>(g.k + kv_row(g, block, h) * (64 * D) + ((unit & ~63) | t) * 16);
  };
  const auto load_v = [&](int block, int u) {
    vr[u] = *reinterpret_cast<const u32x4*>(g.v + kv_row(g, block, h) * (64 * D) + (tid + 256 * u) * 16);
  };
  // 8 of a unit's 16 codes, widened
  const auto put_k = [&](int buf, int u, int part) {
    const int unit = tid + 256 * u;
    sk[buf][2 * (unit >> 6) + part][unit & 63] = codes8(kr[u][2 * part], kr[u][2 * part + 1]);
  };
  const auto put_v = [&](int buf, int u, int part) {
    const int unit = tid + 256 * u;
    sv[buf][2 * (unit / D) + part][unit % D] = codes8(vr[u][2 * part], vr[u][2 * part + 1]);
  };
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = f32x16{};
  float m_run = kLowest, l_run = 0.0f;
  int ev_cur = 0;

  // S^T of the first or second half of the block in sk[buf]
  const auto first_product = [&](f32x16& s, int buf, int u) {
    s = f32x16{};
#pragma unroll
    for (int i = 0; i < NK; ++i) {
      const half8_t kf = sk[buf][2 * i + half][32 * u + col];
      s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, qh[i], s, 0, 0, 0);
      if constexpr (F32) s = __builtin_amdgcn_mfma_f32_32x32x16_f16(kf, ql[i], s, 0, 0, 0);
    }
  };
  const auto second_product = [&](const u32x4 (&ph)[2], const u32x4 (&pl)[2], int buf, int u) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
#pragma unroll
      for (int d = 0; d < ND; ++d) {
        const half8_t vf = sv[buf][4 * u + 2 * i + half][32 * d + col];
        o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, as_half8(ph[i]), o[d], 0, 0, 0);
        if constexpr (F32) o[d] = __builtin_amdgcn_mfma_f32_32x32x16_f16(vf, as_half8(pl[i]), o[d], 0, 0, 0);
      }
  };
  // Masks of scores s (half u of block j), where the block may reach past a row's tokens.
  const auto mask = [&](f32x16& s, int j, int u) {
    if (j * 64 + 32 * u + 32 > lim_lo) {
      const int left = lim - j * 64 - 32 * u - 8 * half;  // result i is token 16 (i / 8) + 8 half + i % 8
#pragma unroll
      for (int i = 0; i < 16; ++i)
        if (16 * (i / 8) + i % 8 >= left) s[i] = -INFINITY;
    }
  };
  const auto rescale = [&](float f) {
#pragma unroll
    for (int d = 0; d < ND; ++d)
#pragma unroll
      for (int i = 0; i < 16; ++i) o[d][i] *= f;
  };
  // After a step: probabilities in terms of an m that a row has left far behind do not
  // fit f16. Their sum shows it (it is over kMost before any of them is over what f16
  // holds), so no maximum is taken until then: m becomes the row's maximum, and the
  // half's probabilities are computed again.
  const auto settle = [&](const f32x16& s, u32x4 (&ph)[2], u32x4 (&pl)[2], float& sum, float ck, int delta) {
    if (!__any(sum > kMost)) return;
    float top = fmaxf(s[0], s[1]);
#pragma unroll
    for (int i = 2; i < 16; ++i) top = fmaxf(top, s[i]);
    const float m_new = fmaxf(m_run, max_halves(top) * ck), alpha = exp2_fast(m_run - m_new);
    l_run *= alpha;
    m_run = m_new;
    rescale(alpha);
    const float off = kBias + (float)delta - m_run;
    float p[16];
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) p[i] = exp2_fast(fmaf(s[i], ck, off));
#pragma unroll
    for (int i = 0; i < 16; ++i) take_p<F32>(p, i, sum, ph, pl);
  };
  // One half block: the softmax of scores s into ph, pl; the second product of the
  // half before (qh_, ql_: its p; vbuf, vu: its V); the first product of the half
  // after (into sn, from kbuf, ku); where `put` says so, the staging of the next
  // block; and at the end, after `between`, the first reads of the next step (nbuf,
  // nu). Written out in the order in which it is to run, one matrix instruction at
  // a time with its share of the rest, and kept so: left to itself the compiler puts
  // all matrix instructions first, each waiting for its own LDS read, and the softmax
  // after them.
  constexpr int SLOTS = 2 * NK, AHEAD = 4, PER = 16 / SLOTS;
  half8_t first[AHEAD];  // operands of a step's first matrix instructions, read in the step before
  const auto step = [&](const f32x16& s, u32x4 (&ph)[2], u32x4 (&pl)[2], const u32x4 (&oh)[2],
                        const u32x4 (&ol)[2], int vbuf, int vu, f32x16& sn, int kbuf, int ku, float ck, int delta,
                        float& sum, int nbuf, int nu, auto put, auto between) {
    static_assert(NK == 2 * ND, "as many matrix instructions for the first product as for the second");
    const auto operand = [&](int i) {
      return i < NK ? sk[kbuf][2 * i + half][32 * ku + col]
                    : sv[vbuf][4 * vu + 2 * ((i - NK) / ND) + half][32 * ((i - NK) % ND) + col];
    };
    const float off = kBias + (float)delta - m_run;
    half8_t in[SLOTS];
    float p[16];
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) in[i] = first[i];
    sn = f32x16{};
#pragma unroll
    for (int i = 0; i < SLOTS; ++i) {
      if (i + AHEAD < SLOTS) in[i + AHEAD] = operand(i + AHEAD);
      if (i == SLOTS - 2) between();
      if (i >= SLOTS - 2) {
#pragma unroll
        for (int n = (i - SLOTS + 2) * AHEAD / 2; n < (i - SLOTS + 3) * AHEAD / 2; ++n)
          first[n] = sk[nbuf][2 * n + half][32 * nu + col];
      }
      // the first product first: its results are then there when the next step begins
      if (i >= NK) {
        const int k = i - NK;
        o[k % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(in[i], as_half8(oh[k / ND]), o[k % ND], 0, 0, 0);
        if constexpr (F32) o[k % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(in[i], as_half8(ol[k / ND]), o[k % ND], 0, 0, 0);
      } else {
        sn = __builtin_amdgcn_mfma_f32_32x32x16_f16(in[i], qh[i], sn, 0, 0, 0);
        if constexpr (F32) sn = __builtin_amdgcn_mfma_f32_32x32x16_f16(in[i], ql[i], sn, 0, 0, 0);
      }
#pragma unroll
      for (int e = i * PER; e < (i + 1) * PER; ++e) p[e] = exp2_fast(fmaf(s[e], ck, off));
      if (i > 0) {
#pragma unroll
        for (int e = (i - 1) * PER; e < i * PER; ++e) take_p<F32>(p, e, sum, ph, pl);
      }
      if (i < SLOTS - 2) put(i);
      __builtin_amdgcn_sched_barrier(0);
    }
#pragma unroll
    for (int e = 16 - PER; e < 16; ++e) take_p<F32>(p, e, sum, ph, pl);
  };

  Walk walk(g, list, b, h, from, to, 1, lane);
  int block = -1, block1 = -1, block2 = -1, ev = 0, ev1 = 0, ev2 = 0;
  float ks = 0.0f, ks1 = 0.0f, ks2 = 0.0f;
  int j = walk.next(block, ks, ev);
  if (j >= 0) {
    f32x16 sa, sb;
    u32x4 pa[2] = {}, pb[2] = {}, la[2] = {}, lb[2] = {};
    // past the last block the registers are loaded with it again (not used), so that
    // the steps have no branch
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      load_k(block, u);
      load_v(block, u);
    }
#pragma unroll
    for (int u = 0; u < UNITS; ++u) {
      put_k(0, u, 0);
      put_k(0, u, 1);
    }
    for (int i = tid; i < 8 * D; i += 256) sv[1][0][i] = half8_t{};  // the pending product of the first half: zero
    block1 = block;
    int j1 = walk.next(block1, ks1, ev1), buf = 0;
#pragma unroll
    for (int u = 0; u < UNITS; ++u) load_k(block1, u);
    __syncthreads();
    first_product(sa, 0, 0);
#pragma unroll
    for (int i = 0; i < AHEAD; ++i) first[i] = sk[0][2 * i + half][32 + col];
    while (true) {
      const float ck = cq * ks;
      float factor, sum;
      const int delta = enter_block(ev_cur, ev, factor);
      const float back = pow2f(-delta);
      if (j * 64 + 64 > len) {
#pragma unroll
        for (int u = 0; u < UNITS; ++u) vr[u] = keep_codes(vr[u], len - j * 64 - 16 * ((tid + 256 * u) / D));
      }
      // half 2 t. The buffers written here were last read before the previous block's
      // barrier. A register's next load follows its last use: a whole block ahead.
      block2 = block1;
      const int j2 = j1 >= 0 ? walk.next(block2, ks2, ev2) : -1;
      mask(sa, j, 0);
      step(sa, pa, la, pb, lb, buf ^ 1, 1, sb, buf, 1, ck, delta, sum, buf ^ 1, 0, [&](int i) {
        // half a unit in each of 4 * UNITS slots: V, then K; as late as the barrier allows
        // where a block takes little time (D = 64: 824 us for the video share from slot 1,
        // 770 from slot 2), since their loads were issued one block ago
        constexpr int FROM = D == 64 ? 2 : 1;
        static_assert(FROM + 4 * UNITS <= SLOTS - 2 || UNITS == 0, "staged before the barrier");
        const int k = i - FROM, u = k / 2 % UNITS;
        if (k < 0 || k >= 4 * UNITS) return;
        if (k < 2 * UNITS) {
          put_v(buf, u, k % 2);
          if (k % 2) load_v(block1, u);
        } else {
          put_k(buf ^ 1, u, k % 2);
          if (k % 2) load_k(block2, u);
        }
      }, [] { __syncthreads(); });
      if (factor != 1.0f) rescale(factor);
      settle(sa, pa, la, sum, ck, delta);
      l_run = fmaf(sum, back, l_run);
      // half 2 t + 1
      mask(sb, j, 1);
      step(sb, pb, lb, pa, la, buf, 0, sa, buf ^ 1, 0, ck, delta, sum, buf ^ 1, 1, [](int) {}, [] {});
      settle(sb, pb, lb, sum, ck, delta);
      l_run = fmaf(sum, back, l_run);
      if (j1 < 0) break;
      buf ^= 1;
      j = j1; block = block1; ks = ks1; ev = ev1;
      j1 = j2; block1 = block2; ks1 = ks2; ev1 = ev2;
    }
    second_product(pb, lb, buf, 1);
  }
  l_run += __shfl_xor(l_run, 32);
  if (!live) return;
  const float unit = pow2f(ev_cur);
  if (a.splits > 1 && split == 0 && half == 0) a.part_n[((int64_t)b * g.kv_heads + h) * rows + r] = parts;
  if (parts > 1) {
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
// D / 4 lanes a row: out = sum O_s 2^(m_s - m) / sum l_s 2^(m_s - m), parts in order.
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
  x *= l > 0.0f ? 1.0f / l : 0.0f;
  IO* out = (IO*)a.out.data + b * a.out.sb + (int64_t)me.query * a.out.st + me.head * a.out.sh + d0;
  if constexpr (F32)
    *reinterpret_cast<f32x4*>(out) = x;
  else
    *reinterpret_cast<u32x2*>(out) = u32x2{bf16_rne(x.x) | bf16_rne(x.y) << 16, bf16_rne(x.z) | bf16_rne(x.w) << 16};
  if (a.lse && d0 == 0)
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
    const int64_t grid = a.splits * ((rows + 127) / 128) * a.g.kv_heads * a.g.batch;
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
