// Attention over packed sequences, for many query rows, fp32.
//
// fp32 products on the f16 matrix units, which are 8.5 times as fast as those for fp32 (1196 and 141
// TFLOP/s measured): x = 2^e (x1 + x2), x1 and x2 in f16 and e the row's own, so that its largest is
// in [2^14, 2^15): 22 bits of each value down to 2^-17 of it, and to 2^-39 of it below (to 2^-146 in
// all, as e is not under -122). A product is x1 y1 + x1 y2 + x2 y1; x2 y2, under 2^-22 of it, is left out.
//
// The split of K and V is done once for all rows that read them, by a kernel before, into the
// plan's workspace: [K1, K2, V1, V2][key head][token][D], and 2^e of each token's K and V. Values that
// are not finite are 0 there, and their token's 2^e negative: scores of such keys (and of queries
// that hold any) are worked out anew from the inputs, such values are added at the end.
//
// The attention is that of the kernel for bf16 (S^T = K Q^T, O^T = V^T P^T, tiles past the
// registers into two LDS buffers), with p = 2^(S 2^(eq + ek) c - m), of which l is the sum, and
// w = p 2^ev as weights of V's halves: m is raised when a w passes 2^15, to where the largest is 2^8,
// so that w fits f16 and is split like the rest (to 2^-33 of a row's largest). For large scores, and
// values of which a row's are far from 1, m is the largest score alone (see `settle`).
//
// Bound by the matrix units at the clock that the card's power allows (1.8 GHz): 8192 queries over 8192
// keys, 16 heads of 128: 1.45 ms, 379 TFLOP/s of attention, 1.14 PFLOP/s of f16 products (a large one of
// the library: 1.21), the matrix units busy 65 % of the cycles; heads of 64: 0.83 ms, where the splitting
// of the weights (9 vector instructions each) takes as long as the products.
// Three waves of a SIMD and tiles of 32 keys for D = 64 (4444 over 4444, 30 heads: 556 us, two waves
// and 64 keys 585); the factors of a step's keys are read before its products (542; now 515). The products of
// one half of a tile beside the weights of the other, as in the bf16 kernel: 559. On the fp32 matrix
// units, by the kernel for few rows: 1566. What the ends of fp32's range take (factors apart, sums that
// show that weights leave it) does not show in large calls for heads of 128, is 1 % for heads of 64 and 3 %
// of causal prompts in short parts; a wave whose m is the largest score weighs every step twice: 4096
// over 4096, 16 heads of 128, 467 us for 414, of 64 351 for 238.
#include <algorithm>
#include <type_traits>

#include "attn_many.hpp"

namespace rc {
namespace {

constexpr float kMost = 0x1p15f, kAbove = 8.0f;  // log2 of the largest weight after m is raised
constexpr float kFine = 0x1p20f;                 // up to here a score and its rounding differ by 2^-4 at most
constexpr float kNear = 60.0f;                   // p is 2^-60 to 2^60 for the largest scores, a rise of m twice as much
constexpr int kExp = 14, kLeast = -122;  // exponent of a row's largest value; e is not below kLeast
constexpr int kNone = -126;              // of values that are all zero
constexpr int kBias = 27;                // the factor of a key is 2^(e - kBias), so that it does not take a score out of fp32

// log2 of 2^e, or of its negative.
__device__ __forceinline__ float exponent_of(float x) { return (float)((int)(__float_as_uint(x) >> 23 & 255u) - 127); }

// 2^e of a row whose largest finite |x| has these bits, 2^-14 for zeros.
__device__ __forceinline__ int row_exponent(uint32_t top) {
  return top == 0u ? -kExp : max((int)(top >> 23) - 127 - kExp, kLeast);
}
__device__ __forceinline__ float power_of_2(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

// x and y as f16, and what that left of them, in three instructions (the compiler takes five and up).
__device__ __forceinline__ void split_pair(float x, float y, uint32_t& hi, uint32_t& lo) {
  asm volatile("" : "+v"(x), "+v"(y));  // or it takes a factor before it into a second conversion
  hi = __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{x, y}), half2_t));
  asm("v_fma_mixlo_f16 %0, %1, -1.0, %2 op_sel_hi:[1,0,0]" : "=v"(lo) : "v"(hi), "v"(x));
  asm("v_fma_mixhi_f16 %0, %1, -1.0, %2 op_sel:[1,0,0] op_sel_hi:[1,0,0]" : "+v"(lo) : "v"(hi), "v"(y));
}

// ------------------------------------------------------------------ K and V as halves
// D / 8 lanes a row.
template <int D>
__global__ __launch_bounds__(256) void attn_halves_kernel(AttnArgs a) {
  constexpr int LANES = D / 8;
  const int64_t rows = (int64_t)a.kv_heads * a.kv_tokens, i = ((int64_t)blockIdx.x * 256 + threadIdx.x) / LANES;
  const int at = threadIdx.x % LANES, which = blockIdx.y;
  const int64_t row = min(i, rows - 1);  // in the order of the inputs, heads inside of tokens
  const int64_t token = row / a.kv_heads;
  const int h = (int)(row % a.kv_heads);
  const KvRows& in = which ? a.v : a.k;
  const f32x4* p = reinterpret_cast<const f32x4*>((const float*)in.data + token * in.st + (int64_t)h * in.sh + 8 * at);
  float x[8];
#pragma unroll
  for (int e = 0; e < 8; e += 4) {
    const f32x4 y = p[e / 4];
#pragma unroll
    for (int k = 0; k < 4; ++k) x[e + k] = y[k];
  }
  uint32_t top = 0;
  bool odd = false;
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    if (not_finite(x[e])) {
      odd = true;
      x[e] = 0.0f;
    }
    top = max(top, __float_as_uint(x[e]) & 0x7FFFFFFFu);
  }
  top = group_max_u32<LANES>(top);
  const uint32_t group = (threadIdx.x & 63) / LANES * LANES;
  odd = (__ballot(odd) >> group & ((1ull << LANES) - 1)) != 0;
  const int e = which && top == 0u ? kNone : row_exponent(top);
  const float inv = power_of_2(-e);
  u32x4 hi, lo;
#pragma unroll
  for (int k = 0; k < 4; ++k) {
    uint32_t y, z;
    split_pair(x[2 * k] * inv, x[2 * k + 1] * inv, y, z);
    hi[k] = y;
    lo[k] = z;
  }
  if (i >= rows) return;
  const int64_t to = ((2 * which) * rows + (int64_t)h * a.kv_tokens + token) * D + 8 * at;
  *reinterpret_cast<u32x4*>(a.halves + to) = hi;
  *reinterpret_cast<u32x4*>(a.halves + to + rows * D) = lo;
  const float factor = ldexpf(1.0f, which ? e : e - kBias);  // 2^-149 at least
  if (at == 0) a.powers[((int64_t)h * 2 + which) * a.kv_tokens + token] = odd ? -factor : factor;
}

// ------------------------------------------------------------------ attention
template <int D>
__global__ __launch_bounds__(256, D == 64 ? 3 : 2) void attn_many_f32_kernel(AttnArgs a) {
  constexpr int NK = D / 16, ND = D / 32, ROWS = 128;
  constexpr int KEYS = 32;  // of a tile in LDS: 32 or 64
  constexpr int PER = D / 8, ROW = 2 * D, PLANE = KEYS * ROW, BYTES = 4 * PLANE;  // chunks, bytes of a row; bytes of K1, of a tile
  constexpr int STEP = 256 / PER, C = KEYS / STEP;  // rows of a load of all threads, loads of a thread for K1
  __shared__ __align__(1024) char shared[2 * BYTES];
  __shared__ __align__(1024) float powers[2][2][KEYS];  // [buffer][K, V]
  __shared__ int shifts[ROWS], lifts[ROWS];  // used by one wave each; lifts: the power of two that `factor` lacks
  const auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  const uint32_t all = gridDim.x / a.splits, w = blockIdx.x % all;
  const int split = a.splits - 1 - (int)(blockIdx.x / all);
  AttnSeq sq;
  const Place place = place_of(a, w, all, ROWS, sq);
  const int b = uniform(place.b), h = uniform(place.h), r0 = uniform(place.tile) * ROWS;
  if (b < 0) {
    if (a.splits > 1 && split == 0 && threadIdx.x == 0) a.joins[w].w = 0;
    return;
  }
  sq = {uniform(sq.q0), uniform(sq.nq), uniform(sq.k0), uniform(sq.nk)};
  const int rows = sq.nq * a.group;
  const int lim_hi = attn_limit(a, sq, (min(r0 + ROWS, rows) - 1) / a.group);
  const int all_tiles = (lim_hi + kTile - 1) / kTile;
  const int parts = min(max((all_tiles + a.chunk - 1) / a.chunk, 1), a.splits), per = (all_tiles + parts - 1) / parts;
  if (a.splits > 1 && split == 0 && threadIdx.x == 0) a.joins[w] = make_int4(b, h, place.tile, parts > 1 ? parts : 0);
  if (split >= parts) return;
  const int from = min(split * per, all_tiles) * (kTile / KEYS);  // tiles of KEYS, up to `tiles`
  const int tiles = min(min(split * per + per, all_tiles) * (kTile / KEYS), (lim_hi + KEYS - 1) / KEYS);
  const int tid = thread_again(), lane = tid & 63, col = lane & 31, half = lane >> 5, wave = uniform(tid >> 6);

  const int64_t plane = (int64_t)a.kv_heads * a.kv_tokens * D;
  const uint16_t* const halves = a.halves + ((int64_t)h * a.kv_tokens + sq.k0) * D;
  const float* const pows = a.powers + (int64_t)h * 2 * a.kv_tokens + sq.k0;
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)shared;
  const uint32_t lds1 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) float*)&powers[0][0][0];
  const auto stage = [&](int tile, int buffer) {
    if (tile >= tiles) return;
    const int lane = thread_again() & 63, srow = wave * (STEP / 4) + lane / PER;
    const uint32_t k_turned = (uint32_t)((lane % PER) ^ k_turn<D>(srow)) * 16, v_turned = (uint32_t)((lane % PER) ^ v_turn<D>(srow)) * 16;
    const uint32_t to = lds0 + (uint32_t)(buffer * BYTES + wave * (STEP / 4) * ROW);
#pragma unroll
    for (int i = 0; i < C; ++i) {
      const int token = min(tile * KEYS + i * STEP + srow, sq.nk - 1) - tile * KEYS;
      const char* const base = (const char*)(halves + (int64_t)tile * KEYS * D);
#pragma unroll
      for (int p = 0; p < 4; ++p)
        load_lds(to + p * PLANE + i * STEP * ROW, (uint32_t)(token * ROW) + (p < 2 ? k_turned : v_turned), base + p * 2 * plane);
    }
    if (wave < KEYS / 32) {
      const int n = wave * 64 + lane, token = min(tile * KEYS + n % KEYS, sq.nk - 1);
      load_lds_4(lds1 + (uint32_t)(buffer * 2 * KEYS + wave * 64) * 4, pows + (int64_t)(n / KEYS) * a.kv_tokens + token);
    }
  };
  stage(from, 0);

  // rows of this wave, and its queries: operand f has channels 16 f + 8 half + 0..7
  const int r = min(r0 + 32 * wave + col, rows - 1);
  half8_t q1[NK], q2[NK];
  float factor;  // of the scores: the row's 2^e and the plan's
  bool odd_row = false, lifted;
  {
    const float* p = (const float*)a.q.data + (int64_t)(sq.q0 + r / a.group) * a.q.st + (int64_t)(h * a.group + r % a.group) * a.q.sh;
    uint32_t top = 0;
    f32x4 x[NK][2];
#pragma unroll
    for (int f = 0; f < NK; ++f)
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        x[f][k] = *reinterpret_cast<const f32x4*>(p + 16 * f + 8 * half + 4 * k);
#pragma unroll
        for (int e = 0; e < 4; ++e) top = max(top, __float_as_uint(x[f][k][e]) & 0x7FFFFFFFu);
      }
    top = max(top, (uint32_t)__shfl_xor((int)top, 32));
    odd_row = top >= 0x7F800000u;
    const int e = odd_row ? 0 : row_exponent(top);
    const float inv = odd_row ? 0.0f : power_of_2(-e);
    // Queries of 2^115 and more, with the keys' bias, can take it out of fp32: what passes 2^127 is kept apart. And it is
    // not 0 for a small one, as a hidden score, -infinity, times 0 is NaN.
    const int lift = max(e + kBias + (int)exponent_of(a.scale) - 126, 0);
    factor = fmaxf(ldexpf(a.scale, e + kBias - lift), 0x1p-149f);
    if (half == 0) lifts[32 * wave + col] = lift;
    lifted = __any(lift > 0);
#pragma unroll
    for (int f = 0; f < NK; ++f) {
      u32x4 hi, lo;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        uint32_t y, z;
        const f32x4 v = x[f][k / 2];
        const float x0 = odd_row ? 0.0f : v[k % 2 * 2], x1 = odd_row ? 0.0f : v[k % 2 * 2 + 1];
        split_pair(x0 * inv, x1 * inv, y, z);
        hi[k] = y;
        lo[k] = z;
      }
      q1[f] = __builtin_bit_cast(half8_t, hi);
      q2[f] = __builtin_bit_cast(half8_t, lo);
    }
  }
  const bool odd_rows = __any(odd_row), uneven = odd_rows || lifted;
  float m_run = kLowest, l_run = 0.0f;
  float most = kMost;  // -1 when m is the largest score, for some row: outputs are held as 2^-shifts of what they are
  int wave_lo = INT32_MAX, my_tiles = 0;  // keys that all its rows see, tiles that one does
  {
    const int first = r0 + 32 * wave, last = min(first + 32, rows) - 1;
    if (first < rows) {
      wave_lo = attn_limit(a, sq, first / a.group);
      my_tiles = min((attn_limit(a, sq, last / a.group) + KEYS - 1) / KEYS, tiles);
    }
  }
  const int lim = attn_limit(a, sq, r / a.group);
  f32x16 o[ND];
#pragma unroll
  for (int d = 0; d < ND; ++d) o[d] = f32x16{};

  const int vrow = 4 * half + (lane & 15) / 4;
  int k_at = col * ROW + (half ^ k_turn<D>(col)) * 16;
  int v_at = 2 * PLANE + vrow * ROW + ((2 * (lane >> 4 & 1) + (lane & 3) / 2) ^ v_turn<D>(vrow)) * 16 + (lane & 1) * 8;

  const auto key = [&](const char* tile, int f) { return *reinterpret_cast<const half8_t*>(tile + (k_at ^ 32 * f)); };
  const auto value = [&](const char* tile, int at) {
    const char* v = tile + 16 * (at / ND) * ROW + (v_at ^ 64 * (at % ND));
    return __builtin_bit_cast(half8_t, __builtin_shufflevector(read_turned(v), read_turned(v + 8 * ROW), 0, 1, 2, 3, 4, 5, 6, 7));
  };
  const auto hide = [&](f32x16& s, int first) {
    if (first + 32 <= wave_lo) return;
    const int left = min(max(lim - first - 4 * (thread_again() >> 5 & 1), 0), 31);
    const uint32_t seen = (1u << left) - 1u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t on = (uint32_t)((int32_t)(seen << (31 - 8 * (i / 4) - i % 4)) >> 31);
      s[i] = __uint_as_float((__float_as_uint(s[i]) & on) | (0xFF800000u & ~on));
    }
  };
  // Scores of keys, or of rows, that are not finite: from the inputs.
  const auto odd_scores = [&](f32x16& s, int first, uint32_t keys) {
    const int half = thread_again() >> 5 & 1;
    const float* p = (const float*)a.q.data + (int64_t)(sq.q0 + r / a.group) * a.q.st + (int64_t)(h * a.group + r % a.group) * a.q.sh + half * (D / 2);
    for (uint32_t left = odd_rows ? 0xFFFFFFFFu : keys; left; left &= left - 1) {
      const int n = __builtin_ctz(left);
      const float* x = (const float*)a.k.data + (int64_t)(sq.k0 + min(first + n, sq.nk - 1)) * a.k.st + (int64_t)h * a.k.sh + half * (D / 2);
      float dot = 0.0f;
#pragma unroll 1
      for (int d = 0; d < D / 2; ++d) dot = fmaf(p[d], x[d], dot);
      dot = sum_halves(dot);
      const bool mine = (n >> 2 & 1) == half && (odd_row || (keys >> n & 1u));
      const int i0 = n / 8 * 4 + n % 4;
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = mine && i == i0 ? dot : s[i];
    }
  };
  const auto add_strange = [&](int first, uint32_t values) {
    const int half = thread_again() >> 5 & 1;
    for (; values; values &= values - 1) {
      const int token = first + __builtin_ctz(values);
      const float* v = (const float*)a.v.data + (int64_t)(sq.k0 + min(token, sq.nk - 1)) * a.v.st + (int64_t)h * a.v.sh;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const f32x4 y = *reinterpret_cast<const f32x4*>(v + 32 * d + 8 * c + 4 * half);
#pragma unroll
          for (int e = 0; e < 4; ++e) o[d][4 * c + e] += token < lim && not_finite(y[e]) ? y[e] : 0.0f;
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  };
  const auto weigh_all = [&](const f32x16& s, const f32x4 (&fk)[4], const f32x4 (&fv)[4], float& sum, float& heavy, u32x4 (&p1)[2], u32x4 (&p2)[2]) {
    sum = heavy = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {
      float e[4];
#pragma unroll
      for (int k = 0; k < 4; ++k) e[k] = exp2_fast(fmaf(s[i + k] * fabsf(fk[i / 4][k]), factor, -m_run));
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        sum += e[k];
        e[k] *= fabsf(fv[i / 4][k]);
      }
#pragma unroll
      for (int k = 0; k < 4; k += 2) heavy = fmaxf(heavy, fmaxf(e[k], e[k + 1]));
#pragma unroll
      for (int k = 0; k < 4; k += 2) {
        uint32_t y, z;
        split_pair(e[k], e[k + 1], y, z);
        p1[i / 8][(i + k) % 8 / 2] = y;
        p2[i / 8][(i + k) % 8 / 2] = z;
      }
      __builtin_amdgcn_sched_barrier(0);
    }
    heavy = fmaxf(heavy, sum * (kMost * 0x1p-100f));  // weights of tiny values may be small where p would leave fp32
  };
  // Whether m has to rise. Where values are so large or small (or zero) that an m that follows p 2^ev is far from the
  // scores, p or what is left of l when m rises would leave fp32; for large scores fp32 is too coarse for such an m (from
  // 2^27 on none makes all weights fit f16). m is then the largest score, rounded like all of them, and a power of two of
  // the row's own brings its weights into f16.
  const auto settle = [&](const f32x16& s, const f32x4 (&fk)[4], const f32x4 (&fv)[4], float& sum, float heavy, u32x4 (&p1)[2], u32x4 (&p2)[2]) {
    if (__any(heavy > most)) {
      const auto score = [&](int i) { return s[i] * fabsf(fk[i / 4][i % 4]); };  // without the factor
      const auto weight = [&](float t, int i) { return t + exponent_of(fv[i / 4][i % 4]); };  // log2 of it
      float high = -INFINITY, top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const float t = score(i) * factor;
        high = fmaxf(high, t);
        top = fmaxf(top, weight(t, i));
        __builtin_amdgcn_sched_barrier(0);
      }
      high = max_halves(high);
      top = max_halves(top) - kAbove;
      float m_new = fmaxf(m_run, top);
      const bool far = high - kNear > m_new || (top > m_run && top - high > kNear) || (m_run != kLowest && m_new - m_run > 2.0f * kNear);
      const bool was = most != kMost, coarse = was || __any(far || (m_new != kLowest && fabsf(m_new) > kFine));
      most = coarse ? -1.0f : kMost;
      int shift = 0, now = 0;
      if (coarse) {
        int* const at = &shifts[thread_again() / 64 * 32 + (thread_again() & 31)];
        shift = was ? *at : 0;
        m_new = fmaxf(m_run, high);
        top = -INFINITY;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          top = fmaxf(top, weight(score(i) * factor - m_new, i));
          __builtin_amdgcn_sched_barrier(0);
        }
        // 2^13 for the largest weight of these keys, or what is left of the largest before
        now = max((int)fmaxf(max_halves(top), (float)kLeast) - 13, shift + (int)fmaxf(m_run - m_new, -1000.0f));
        *at = now;
      }
      const float down = m_run - m_new, alpha = exp2_fast(down + (float)(shift - now));
      l_run *= exp2_fast(down);
      m_run = m_new;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[d][k] *= alpha;
      const auto weigh_again = [&](auto apart) {
        sum = 0.0f;
#pragma unroll
        for (int i = 0; i < 16; i += 2) {
          float e[2];
#pragma unroll
          for (int k = 0; k < 2; ++k) {
            e[k] = exp2_fast(score(i + k) * factor - m_run);
            sum += e[k];
            const float v = fabsf(fv[i / 4][i % 4 + k]);
            e[k] = decltype(apart)::value ? ldexpf(ldexpf(e[k], -now / 2) * v, -now - -now / 2) : e[k] * v;
          }
          uint32_t hi, lo;
          split_pair(e[0], e[1], hi, lo);
          p1[i / 8][i % 8 / 2] = hi;
          p2[i / 8][i % 8 / 2] = lo;
          __builtin_amdgcn_sched_barrier(0);
        }
      };
      if (coarse) weigh_again(std::true_type{});
      else weigh_again(std::false_type{});
    }
    l_run += sum;
  };
  const auto keys_32 = [&](const char* tile, const float* pow, int first) {
    asm volatile("" : "+v"(k_at), "+v"(v_at));  // or all their forms would be kept in registers
    f32x16 s = {};
    u32x4 p1[2], p2[2];
    float sum, heavy;
    half8_t n1 = key(tile, 0), n2 = key(tile + PLANE, 0);
    f32x4 fk[4], fv[4];  // factors of the keys and values whose scores the lane gets, four and four
    {
      const float* const at = pow + 4 * (thread_again() >> 5 & 1);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        fk[i] = *reinterpret_cast<const f32x4*>(at + 8 * i);
        fv[i] = *reinterpret_cast<const f32x4*>(at + 8 * i + KEYS);
      }
    }
#pragma unroll
    for (int f = 0; f < NK; ++f) {
      const half8_t k1 = n1, k2 = n2;
      if (f + 1 < NK) {
        n1 = key(tile, f + 1);
        n2 = key(tile + PLANE, f + 1);
      }
      s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k2, q1[f], s, 0, 0, 0);
      s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k1, q2[f], s, 0, 0, 0);
      s = __builtin_amdgcn_mfma_f32_32x32x16_f16(k1, q1[f], s, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    const int again = thread_again(), half = again >> 5 & 1;
    const uint64_t odd = __ballot(pow[(again & 31) + half * KEYS] < 0.0f);
    if (uneven || (uint32_t)odd) {
      const int lift = lifts[again / 64 * 32 + (again & 31)];
#pragma unroll
      for (int i = 0; i < 16; ++i) s[i] = ldexpf(s[i], lift);
      if (odd_rows || (uint32_t)odd) odd_scores(s, first, (uint32_t)odd);
    }
    hide(s, first);
    n1 = value(tile, 0);
    n2 = value(tile + PLANE, 0);
    weigh_all(s, fk, fv, sum, heavy, p1, p2);
    settle(s, fk, fv, sum, heavy, p1, p2);
#pragma unroll
    for (int at = 0; at < 2 * ND; ++at) {
      const half8_t v1 = n1, v2 = n2, w1 = __builtin_bit_cast(half8_t, p1[at / ND]), w2 = __builtin_bit_cast(half8_t, p2[at / ND]);
      if (at + 1 < 2 * ND) {
        n1 = value(tile, at + 1);
        n2 = value(tile + PLANE, at + 1);
      }
      o[at % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v2, w1, o[at % ND], 0, 0, 0);
      o[at % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, w2, o[at % ND], 0, 0, 0);
      o[at % ND] = __builtin_amdgcn_mfma_f32_32x32x16_f16(v1, w1, o[at % ND], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (odd >> 32) add_strange(first, (uint32_t)(odd >> 32));
  };

  wait_loads();
  for (int t = from; t < tiles; ++t) {
    const int buffer = (t - from) & 1;
    wait_loads();     // this wave's of tile t are in LDS
    __syncthreads();  // the others' too, and the last tile is read
    stage(t + 1, 1 - buffer);
    if (t >= my_tiles) continue;
    const char* const tile = shared + buffer * BYTES;
#pragma unroll
    for (int k = 0; k < KEYS; k += 32) keys_32(tile + k * ROW, &powers[buffer][0][k], t * KEYS + k);
  }

  const int64_t slot = (int64_t)w * a.splits + split;  // of partial results
  const int again = thread_again(), lane_ = again & 63, half_ = lane_ >> 5, row = r0 + 32 * wave + (lane_ & 31);
  float l = sum_halves(l_run), inv = attn_inverse(l);
  if (most != kMost) {
    const int shift = shifts[32 * wave + (lane_ & 31)];
    if (parts > 1) {  // the power goes into m, as far as m has the bits, or a sum of large values could leave fp32
      const float m = m_run + fmaxf((float)shift, -kNear), by = m_run - m, root = exp2_fast(0.5f * ((float)shift + by));
      m_run = m;
      l *= exp2_fast(by);
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[d][k] = o[d][k] * root * root;
    } else {
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[d][k] = ldexpf(o[d][k] * inv, shift);
    }
  }
  const float last = parts > 1 || most != kMost ? 1.0f : inv;
  f32x4* const part = reinterpret_cast<f32x4*>(a.part) + (slot * (ROWS / 32) + wave) * ND * 4 * 64 + lane_;
  const int query = sq.q0 + row / a.group, head = h * a.group + row % a.group;
  const bool live = row < rows;
  float* const out = (float*)a.out.data + (int64_t)query * a.out.st + (int64_t)head * a.out.sh + 4 * half_;
#pragma unroll
  for (int d = 0; d < ND; ++d)
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      f32x4 x;
#pragma unroll
      for (int e = 0; e < 4; ++e) x[e] = o[d][4 * c + e];
      if (parts > 1) part[(d * 4 + c) * 64] = x;  // as the lanes hold them
      else if (live) *reinterpret_cast<f32x4*>(out + 32 * d + 8 * c) = x * last;
    }
  if (live && half_ == 0) {
    if (parts > 1) a.part_ml[slot * ROWS + 32 * wave + lane_] = make_float2(m_run, l);
    else if (a.lse) a.lse[(int64_t)query * a.q_heads + head] = attn_lse(m_run, l);
  }
}

template <int D>
hipError_t run(const AttnArgs& a, int64_t grid, hipStream_t s) {
  const int64_t blocks = ((int64_t)a.kv_heads * a.kv_tokens * (D / 8) + 255) / 256;
  if (grid > INT32_MAX || blocks > INT32_MAX) return hipErrorInvalidValue;
  if (blocks) attn_halves_kernel<D><<<dim3((unsigned)blocks, 2), 256, 0, s>>>(a);
  hipError_t err = hipGetLastError();
  if (err != hipSuccess) return err;
  attn_many_f32_kernel<D><<<(unsigned)grid, 256, 0, s>>>(a);
  err = hipGetLastError();
  if (err == hipSuccess && a.splits > 1) {
    attn_many_join_kernel<D, 128, true><<<(unsigned)(grid / a.splits) * (D / 32), 256, 0, s>>>(a);
    err = hipGetLastError();
  }
  return err;
}

}  // namespace

hipError_t launch_attn_many_f32(const AttnArgs& a, int64_t grid, hipStream_t s) {
  return a.dim == 64 ? run<64>(a, grid, s) : run<128>(a, grid, s);
}

}  // namespace rc
