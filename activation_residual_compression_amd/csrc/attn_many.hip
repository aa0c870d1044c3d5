// Attention over packed sequences, for many query rows, bf16.
//
// One block of threads: 128 U rows of one key head of one sequence (row r: query r / G, query head
// h * G + r % G), a part of the keys. KG groups of four waves have the same rows, 32 U a wave, and
// take every KG-th tile of 64 keys. A group's tiles go through two LDS buffers of 64 D x 4 bytes,
// written past the registers while the other is read; one barrier a tile. Groups are joined in
// LDS, parts by a second launch.
//
// S^T = K Q^T and O^T = V^T P^T: a lane holds scores of one row only (its column), the softmax
// is in the lane, and its weights, rounded to bf16, are the second product's operand as they
// are: result i of the first lies at key 8 (i / 4) + 4 half + i % 4, so lane half `half` holds
// keys 16 m + 4 half + 0..3 and 16 m + 8 + 4 half + 0..3 for step m of the second product, and V
// is read in that order, transposed four keys at a time by the LDS's own transposing read.
//
// Softmax in base 2, p = 2^(S c - m). m is not the running maximum: it is raised only when the
// weights of a step sum to more than 2^10, which the sum shows that is needed anyway, so the
// accumulators are rescaled a few times in all, and no maximum is taken otherwise. bf16 and
// fp32 hold such weights as well as those up to 1; both cancel in out = O / l. m is S c rounded:
// past 2^20 the weights take the same rounding, or their difference would leave fp32 (from 2^30 on).
// Such a wave weighs every step twice: 4096 over 4096, 16 heads of 128, 184 us for 129.
//
// Weights as one bf16, half a step of 2^-8 each: against 64 bits the outputs are off by 0.0021 to
// 0.0023 of their norm, 0.0016 to 0.0017 by their own rounding alone. As two bf16 (16 bits, like the
// kernel for few rows, which waits for memory) the second product takes twice as many matrix
// instructions where these bound the kernel: 8192 over 8192, 32 / 8 heads of 128, 1366 us for 911; 4444
// over 17776, 30 heads of 64, 985 for 662; causal ragged prompts, 16 / 4 heads of 128, 174 for 111.
//
// Bound by the matrix units and the power they may draw: a tile of 64 keys of a wave with 64 rows is
// 64 (D 128) matrix instructions of 32 cycles, beside which run 64 weights a lane (a multiply-add, an
// exponential, an addition, half a conversion each) and the LDS reads. 8192 queries over 8192 keys, 32
// heads of 128 on 8: 896 us, 1227 TFLOP/s (a large matrix product of the library: 1251), the matrix units
// 62 % busy at the 1.7 GHz that the card's power allows; at 64 channels 50 %, the vector units 72 %:
// 4444 over 17776, 30 heads of 64: 650 us, 933 TFLOP/s. U = 2 reads K and V from LDS once for 64
// rows: with one row group a wave LDS bounds it (1087 us). KG = 2 is for calls of few tiles of
// rows, where a CU would hold one block of four waves: 1152 over 4608, 2 x 24 heads of 128, 126
// us, KG = 1 171.
#include <algorithm>
#include <type_traits>

#include "attn_many.hpp"

namespace rc {
namespace {

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
constexpr float kMost = 0x1p10f;
constexpr float kFine = 0x1p20f;  // up to here S c and its rounding differ by 2^-4 at most

template <int D, int U, int KG>
__global__ __launch_bounds__(256 * KG, 2) void attn_many_kernel(AttnArgs a) {
  constexpr int NK = D / 16, ND = D / 32, ROWS = 128 * U;
  constexpr int PER = D / 8, ROW = 2 * D, HALF = kTile * ROW, BYTES = 2 * HALF;  // chunks, bytes of a row; bytes of K, of a tile
  constexpr int C = D / 32, STEP = kTile / C;  // loads of a thread for a tile of K, and the rows between two of them
  __shared__ __align__(1024) char shared[KG * 2 * BYTES];
  __shared__ float2 sml[KG == 1 ? 1 : 2][KG == 1 ? 1 : ROWS];
  __shared__ int strange[KG];  // a group's last tile that held a value which is not finite and hidden from some row
  const auto uniform = [](int x) { return __builtin_amdgcn_readfirstlane(x); };
  // The last parts of all tiles come first: only the long tiles have such.
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
  const int lim_lo = attn_limit(a, sq, r0 / a.group);
  const int lim_hi = attn_limit(a, sq, (min(r0 + ROWS, rows) - 1) / a.group);
  const int all_tiles = (lim_hi + kTile - 1) / kTile;
  const int parts = min(max((all_tiles + a.chunk - 1) / a.chunk, 1), a.splits), per = (all_tiles + parts - 1) / parts;
  if (a.splits > 1 && split == 0 && threadIdx.x == 0) a.joins[w] = make_int4(b, h, place.tile, parts > 1 ? parts : 0);
  if (split >= parts) return;
  const int from = min(split * per, all_tiles), tiles = min(from + per, all_tiles);  // up to `tiles`
  const int tid = thread_again(), lane = tid & 63, col = lane & 31, half = lane >> 5;
  const int wave = uniform(tid >> 6) & 3, group = KG == 1 ? 0 : uniform(tid >> 8);
  char* const mine = shared + group * 2 * BYTES;

  // staging: load i of a thread has chunk lane % PER of row STEP i + srow, whose turn does not depend on i
  const char* const kh = (const char*)((const uint16_t*)a.k.data + (int64_t)sq.k0 * a.k.st + (int64_t)h * a.k.sh);
  const char* const vh = (const char*)((const uint16_t*)a.v.data + (int64_t)sq.k0 * a.v.st + (int64_t)h * a.v.sh);
  const uint32_t lds0 = (uint32_t)(uintptr_t)(__attribute__((address_space(3))) char*)mine;
  const bool near = (a.k.st | a.v.st) < (int64_t)1 << 24;  // a tile's offsets fit 32 bits
  const auto stage = [&](int tile, int buffer) {
    if (tile >= tiles) return;
    const int lane = thread_again() & 63, srow = wave * (STEP / 4) + lane / PER;
    const uint32_t k_turned = (uint32_t)((lane % PER) ^ k_turn<D>(srow)) * 16, v_turned = (uint32_t)((lane % PER) ^ v_turn<D>(srow)) * 16;
    const uint32_t to = lds0 + (uint32_t)(buffer * BYTES + wave * (STEP / 4) * ROW);
    if (near && (tile + 1) * kTile <= sq.nk) {
      const uint32_t k_off = (uint32_t)srow * (uint32_t)(2 * a.k.st) + k_turned, v_off = (uint32_t)srow * (uint32_t)(2 * a.v.st) + v_turned;
#pragma unroll
      for (int i = 0; i < C; ++i) {
        load_lds(to + i * STEP * ROW, k_off, kh + (int64_t)(tile * kTile + i * STEP) * (2 * a.k.st));
        load_lds(to + HALF + i * STEP * ROW, v_off, vh + (int64_t)(tile * kTile + i * STEP) * (2 * a.v.st));
      }
    } else {
#pragma unroll 1
      for (int i = 0; i < C; ++i) {
        const int64_t token = min(tile * kTile + i * STEP + srow, sq.nk - 1);
        load_lds(to + i * STEP * ROW, kh + token * (2 * a.k.st) + k_turned);
        load_lds(to + HALF + i * STEP * ROW, vh + token * (2 * a.v.st) + v_turned);
      }
    }
  };
  stage(from + group, 0);

  // rows of this wave, and its queries: operand f has channels 16 f + 8 half + 0..7
  bf16x8 q[U][NK];
  float m_run[U], l_run[U];
  float most = kMost;  // -1 when some row's m is past kFine
  int wave_lo = INT32_MAX, my_tiles = 0;  // keys that all its rows see, tiles that one does
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int r = min(r0 + 32 * U * wave + 32 * u + col, rows - 1);
    const uint16_t* p = (const uint16_t*)a.q.data + (int64_t)(sq.q0 + r / a.group) * a.q.st + (int64_t)(h * a.group + r % a.group) * a.q.sh;
#pragma unroll
    for (int f = 0; f < NK; ++f) q[u][f] = *reinterpret_cast<const bf16x8*>(p + 16 * f + 8 * half);
    m_run[u] = kLowest;
    l_run[u] = 0.0f;
  }
  {
    const int first = r0 + 32 * U * wave, last = min(first + 32 * U, rows) - 1;
    if (first < rows) {
      wave_lo = attn_limit(a, sq, first / a.group);
      my_tiles = min((attn_limit(a, sq, last / a.group) + kTile - 1) / kTile, tiles);
    }
  }
  const auto limit = [&](int u) {  // keys that the lane's row sees
    return attn_limit(a, sq, min(r0 + 32 * U * wave + 32 * u + (thread_again() & 31), rows - 1) / a.group);
  };
  f32x16 o[U][ND];
#pragma unroll
  for (int u = 0; u < U; ++u)
#pragma unroll
    for (int d = 0; d < ND; ++d) o[u][d] = f32x16{};

  // places of the operands in a tile: row part + (chunk part ^ 32 f), (^ 64 d)
  const int vrow = 4 * half + (lane & 15) / 4;
  int k_at = col * ROW + (half ^ k_turn<D>(col)) * 16;
  int v_at = HALF + vrow * ROW + ((2 * (lane >> 4 & 1) + (lane & 3) / 2) ^ v_turn<D>(vrow)) * 16 + (lane & 1) * 8;

  // operand f of K of the 32 keys whose rows begin at `tile`, and of their V: step at / ND of channels 32 (at % ND)
  const auto key = [&](const char* tile, int f) { return *reinterpret_cast<const bf16x8*>(tile + (k_at ^ 32 * f)); };
  const auto value = [&](const char* tile, int at) {
    const char* v = tile + 16 * (at / ND) * ROW + (v_at ^ 64 * (at % ND));
    return __builtin_bit_cast(bf16x8, __builtin_shufflevector(read_turned(v), read_turned(v + 8 * ROW), 0, 1, 2, 3, 4, 5, 6, 7));
  };
  const auto hide = [&](f32x16& s, int u, int first) {  // scores of keys from `first` on that the row does not see
    if (first + 32 <= wave_lo) return;
    // by bits, not by comparisons, whose 16 results at once would spill scalars
    const int left = min(max(limit(u) - first - 4 * (thread_again() >> 5 & 1), 0), 31);  // the last bit, key 28, is the highest used
    const uint32_t seen = (1u << left) - 1u;
#pragma unroll
    for (int i = 0; i < 16; ++i) {
      const uint32_t on = (uint32_t)((int32_t)(seen << (31 - 8 * (i / 4) - i % 4)) >> 31);
      s[i] = __uint_as_float((__float_as_uint(s[i]) & on) | (0xFF800000u & ~on));
    }
  };
  // weights i .. i + N - 1 of 32 keys
  const auto weigh = [&](const f32x16& s, int u, int i, auto n, float& sum, u32x4 (&p)[2]) {
    constexpr int N = decltype(n)::value;
    float e[N];
#pragma unroll
    for (int k = 0; k < N; ++k) e[k] = exp2_fast(fmaf(s[i + k], a.scale, -m_run[u]));
#pragma unroll
    for (int k = 0; k < N; ++k) sum += e[k];
#pragma unroll
    for (int k = 0; k < N; k += 2) {
      uint32_t w = bf16_pair(e[k], e[k + 1]);
      asm volatile("" : "+v"(w), "+v"(sum));  // in its place, or the compiler gathers all at the end
      p[(i + k) / 8][(i + k) % 8 / 2] = w;
    }
  };
  // The same with S c rounded like m: from 2^30 on their difference would take the weights out of fp32.
  const auto weigh_rounded = [&](const f32x16& s, int u, float& sum, u32x4 (&p)[2]) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 2) {
      const float x = exp2_fast(s[i] * a.scale - m_run[u]), y = exp2_fast(s[i + 1] * a.scale - m_run[u]);
      sum += x + y;
      p[i / 8][i % 8 / 2] = bf16_pair(x, y);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const auto weigh_all = [&](const f32x16& s, int u, float& sum, u32x4 (&p)[2]) {
    sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; i += 4) {  // four at a time, so that they take few registers
      weigh(s, u, i, std::integral_constant<int, 4>{}, sum, p);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  const auto settle = [&](const f32x16& s, int u, float& sum, u32x4 (&p)[2]) {  // whether m has to rise
    if (__any(!(sum <= most))) {
      float top = s[0];
#pragma unroll
      for (int i = 1; i < 16; ++i) top = fmaxf(top, s[i]);
      const float m_new = fmaxf(m_run[u], max_halves(top) * a.scale), alpha = exp2_fast(m_run[u] - m_new);
      l_run[u] *= alpha;
      m_run[u] = m_new;
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int k = 0; k < 16; ++k) o[u][d][k] *= alpha;
      const bool coarse = most != kMost || __any(fabsf(m_new) > kFine && m_new != kLowest);
      most = coarse ? -1.0f : kMost;
      if (coarse) weigh_rounded(s, u, sum, p);
      else weigh_all(s, u, sum, p);
    }
    l_run[u] += sum;
  };
  // A tile of keys. Two row groups: operands of K and V serve both, 32 keys at a time.
  const auto shared_keys = [&](const char* tile, int first) {
    asm volatile("" : "+v"(k_at), "+v"(v_at));  // or all their forms would be kept in registers
    f32x16 s[U] = {};
    u32x4 p[U][2];
    float sum;
    bf16x8 next = key(tile, 0);
    if constexpr (D == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int f = 0; f < NK; ++f) {
      const bf16x8 now = next;
      if (f + 1 < NK) next = key(tile, f + 1);
#pragma unroll
      for (int u = 0; u < U; ++u) s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now, q[u][f], s[u], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (D == 128) __builtin_amdgcn_s_setprio(0);
#pragma unroll
    for (int u = 0; u < U; ++u) hide(s[u], u, first);
    next = value(tile, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      weigh_all(s[u], u, sum, p[u]);
      settle(s[u], u, sum, p[u]);
    }
    if constexpr (D == 128) __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int at = 0; at < 2 * ND; ++at) {
      const bf16x8 now = next;
      if (at + 1 < 2 * ND) next = value(tile, at + 1);
#pragma unroll
      for (int u = 0; u < U; ++u)
        o[u][at % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now, __builtin_bit_cast(bf16x8, p[u][at / ND]), o[u][at % ND], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    if constexpr (D == 128) __builtin_amdgcn_s_setprio(0);
  };
  // One row group: the tile's two halves, the products of one beside the softmax of the other, two or four weights to
  // a matrix instruction (8192 queries over 8192 keys, 16 heads of 128: 528 us, one after the other 543).
  const auto in_turn = [&](const char* tile, int first) {
    asm volatile("" : "+v"(k_at), "+v"(v_at));
    const char* const tile_b = tile + 32 * ROW;
    f32x16 sa = {}, sb = {};
    u32x4 pa[2], pb[2];
    float suma = 0.0f, sumb = 0.0f;
    bf16x8 next = key(tile, 0);
#pragma unroll
    for (int f = 0; f < NK; ++f) {
      const bf16x8 now = next;
      next = f + 1 < NK ? key(tile, f + 1) : key(tile_b, 0);
      sa = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now, q[0][f], sa, 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
    hide(sa, 0, first);
#pragma unroll
    for (int f = 0; f < NK; ++f) {
      sb = __builtin_amdgcn_mfma_f32_32x32x16_bf16(next, q[0][f], sb, 0, 0, 0);
      if (f + 1 < NK) next = key(tile_b, f + 1);
      weigh(sa, 0, 16 / NK * f, std::integral_constant<int, 16 / NK>{}, suma, pa);
      __builtin_amdgcn_sched_barrier(0);
    }
    settle(sa, 0, suma, pa);
    hide(sb, 0, first + 32);
    next = value(tile, 0);
#pragma unroll
    for (int at = 0; at < 2 * ND; ++at) {
      o[0][at % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(next, __builtin_bit_cast(bf16x8, pa[at / ND]), o[0][at % ND], 0, 0, 0);
      next = at + 1 < 2 * ND ? value(tile, at + 1) : value(tile_b, 0);
      weigh(sb, 0, 8 / ND * at, std::integral_constant<int, 8 / ND>{}, sumb, pb);
      __builtin_amdgcn_sched_barrier(0);
    }
    settle(sb, 0, sumb, pb);
#pragma unroll
    for (int at = 0; at < 2 * ND; ++at) {
      const bf16x8 now = next;
      if (at + 1 < 2 * ND) next = value(tile_b, at + 1);
      o[0][at % ND] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(now, __builtin_bit_cast(bf16x8, pb[at / ND]), o[0][at % ND], 0, 0, 0);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // What is not finite among values that some row does not see is taken out of the product
  // (zero times it is NaN) and added after it for the rows that see it.
  const auto clear = [&](int t, char* tile) {
    const int lane = thread_again() & 63, srow = wave * (STEP / 4) + lane / PER;
    bool odd = false;
#pragma unroll 1
    for (int i = 0; i < C; ++i) {
      const int row = i * STEP + srow;
      u32x4* at = reinterpret_cast<u32x4*>(tile + HALF + row * ROW + lane % PER * 16);
      u32x4 x = *at;
      bool here = false;
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        const bool lo = (x[w] & 0x7F80u) == 0x7F80u, hi = (x[w] & 0x7F800000u) == 0x7F800000u;
        here |= lo || hi;
        x[w] = lo ? x[w] & 0xFFFF0000u : x[w];
        x[w] = hi ? x[w] & 0xFFFFu : x[w];
      }
      if (here && t * kTile + row >= lim_lo) {
        *at = x;
        odd = true;
      }
    }
    if (odd) strange[group] = t;
  };
  const auto add_strange = [&](int t) {
    const int half = thread_again() >> 5 & 1;
    int lim[U];
#pragma unroll
    for (int u = 0; u < U; ++u) lim[u] = limit(u);
    for (int token = max(t * kTile, lim_lo); token < min((t + 1) * kTile, lim_hi); ++token) {
      const uint16_t* v = (const uint16_t*)(vh + token * (2 * a.v.st));
#pragma unroll
      for (int d = 0; d < ND; ++d)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          const u32x2 w = *reinterpret_cast<const u32x2*>(v + 32 * d + 8 * c + 4 * half);
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float y = e % 2 ? bf16_hi(w[e / 2]) : bf16_lo(w[e / 2]);
            const float add = not_finite(y) ? y : 0.0f;
#pragma unroll
            for (int u = 0; u < U; ++u) o[u][d][4 * c + e] += token < lim[u] ? add : 0.0f;
          }
          __builtin_amdgcn_sched_barrier(0);
        }
    }
  };

  if (thread_again() < KG) strange[thread_again()] = from - 1;
  wait_loads();
  for (int n = from; n < tiles; n += KG) {
    const int t = n + group;
    char* const tile = mine + ((n - from) / KG & 1) * BYTES;
    wait_loads();     // this wave's of tile t are in LDS
    __syncthreads();  // the others' too, and the last tile is read
    stage(t + KG, ~((n - from) / KG) & 1);
    if ((n + KG) * kTile > lim_lo) {
      if (t < tiles) clear(t, tile);
      __syncthreads();
    }
    if (t >= my_tiles) continue;
    if constexpr (U == 1) {
      in_turn(tile, t * kTile);
    } else {
      shared_keys(tile, t * kTile);
      shared_keys(tile + 32 * ROW, t * kTile + 32);
    }
    if (strange[group] == t) add_strange(t);
  }

  const int64_t slot = (int64_t)w * a.splits + split;  // of partial results
  const int again = thread_again(), lane_ = again & 63, half_ = lane_ >> 5, row0 = 32 * U * wave + (lane_ & 31);
#pragma unroll
  for (int u = 0; u < U; ++u) l_run[u] = sum_halves(l_run[u]);
  // With two groups either keeps half of the channels and hands over the others.
  constexpr int NO = ND / KG;
  f32x4* const give = reinterpret_cast<f32x4*>(shared + (KG - 1 - group) * (2 * BYTES)) + wave * (U * NO * 4 * 64) + lane_;
  const f32x4* const take = reinterpret_cast<const f32x4*>(mine) + wave * (U * NO * 4 * 64) + lane_;
  __syncthreads();  // LDS is read
  if constexpr (KG == 2) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      if (half_ == 0) sml[group][row0 + 32 * u] = make_float2(m_run[u], l_run[u]);
#pragma unroll
      for (int d = 0; d < NO; ++d)
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          f32x4 x;
#pragma unroll
          for (int e = 0; e < 4; ++e) x[e] = group ? o[u][d][4 * c + e] : o[u][NO + d][4 * c + e];
          give[((u * NO + d) * 4 + c) * 64] = x;
        }
    }
    __syncthreads();
  }
#pragma unroll
  for (int u = 0; u < U; ++u) {
    float m = m_run[u], l = l_run[u], f = 1.0f, g = 0.0f;
    if constexpr (KG == 2) {
      const float2 other = sml[1 - group][row0 + 32 * u];
      m = fmaxf(m_run[u], other.x);
      f = exp2_fast(m_run[u] - m);
      g = exp2_fast(other.x - m);
      l = l_run[u] * f + other.y * g;
    }
    const int r = r0 + row0 + 32 * u;
    const bool live = r < rows;
    f32x4* const part = reinterpret_cast<f32x4*>(a.part) + ((slot * (ROWS / 32) + wave * U + u) * ND + group * NO) * 4 * 64 + lane_;
    const float inv = attn_inverse(l);
    const int query = sq.q0 + r / a.group, head = h * a.group + r % a.group;
    uint16_t* const out = (uint16_t*)a.out.data + (int64_t)query * a.out.st + (int64_t)head * a.out.sh + group * (D / 2) + 8 * half_;
#pragma unroll
    for (int d = 0; d < NO; ++d)
#pragma unroll
      for (int c = 0; c < 4; c += 2) {
        f32x4 x[2];
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int e = 0; e < 4; ++e) x[k][e] = KG == 2 && group ? o[u][ND - NO + d][4 * (c + k) + e] : o[u][d][4 * (c + k) + e];
        if constexpr (KG == 2) {
#pragma unroll
          for (int k = 0; k < 2; ++k) x[k] = x[k] * f + take[((u * NO + d) * 4 + c + k) * 64] * g;
        }
        if (parts > 1) {  // as the lanes hold them
          part[(d * 4 + c) * 64] = x[0];
          part[(d * 4 + c + 1) * 64] = x[1];
        } else {
          const u32x4 w = rows_of_8(x[0] * inv, x[1] * inv);
          if (live) *reinterpret_cast<u32x4*>(out + 32 * d + 8 * c) = w;
        }
      }
    if (live && group == 0 && half_ == 0) {
      if (parts > 1) a.part_ml[slot * ROWS + row0 + 32 * u] = make_float2(m, l);
      else if (a.lse) a.lse[(int64_t)query * a.q_heads + head] = attn_lse(m, l);
    }
  }
}

template <int D, int U, int KG>
hipError_t run(const AttnArgs& a, int64_t grid, hipStream_t s) {
  if (grid > INT32_MAX) return hipErrorInvalidValue;
  attn_many_kernel<D, U, KG><<<(unsigned)grid, 256 * KG, 0, s>>>(a);
  hipError_t err = hipGetLastError();
  if (err == hipSuccess && a.splits > 1) {
    attn_many_join_kernel<D, 128 * U, false><<<(unsigned)(grid / a.splits) * (U * D / 32), 256, 0, s>>>(a);
    err = hipGetLastError();
  }
  return err;
}

template <int D>
hipError_t pick(const AttnArgs& a, int u, int kg, int64_t grid, hipStream_t s) {
  if (kg == 1) return u == 1 ? run<D, 1, 1>(a, grid, s) : run<D, 2, 1>(a, grid, s);
  return u == 1 ? run<D, 1, 2>(a, grid, s) : run<D, 2, 2>(a, grid, s);
}

}  // namespace

hipError_t launch_attn_many(const AttnArgs& a, int u, int kg, int64_t grid, hipStream_t s) {
  return a.dim == 64 ? pick<64>(a, u, kg, grid, s) : pick<128>(a, u, kg, grid, s);
}

}  // namespace rc
