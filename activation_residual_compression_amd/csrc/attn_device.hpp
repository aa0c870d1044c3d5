// Device helpers of attention over packed sequences.
#pragma once

#include "attn.hpp"
#include "kv_device.hpp"

namespace rc {

// A sequence of the call: its first query and key token, and how many it has.
struct AttnSeq {
  int q0, nq, k0, nk;
};
__device__ __forceinline__ AttnSeq attn_seq(const AttnArgs& a, int b) {
  const int q0 = min(max(a.q_off[b], 0), a.q_tokens), q1 = min(a.q_off[b + 1], a.q_tokens);
  const int k0 = min(max(a.kv_off[b], 0), a.kv_tokens), k1 = min(a.kv_off[b + 1], a.kv_tokens);
  return {q0, min(max(q1 - q0, 0), a.max_q), k0, min(max(k1 - k0, 0), a.max_kv)};
}
// Queries of sequence b.
__device__ __forceinline__ int attn_queries(const AttnArgs& a, int b) {
  const int q0 = min(max(a.q_off[b], 0), a.q_tokens), q1 = min(a.q_off[b + 1], a.q_tokens);
  return min(max(q1 - q0, 0), a.max_q);
}
// Keys that query i of the sequence sees.
__device__ __forceinline__ int attn_limit(const AttnArgs& a, const AttnSeq& s, int i) {
  return a.causal ? max(0, s.nk - s.nq + i + 1) : s.nk;
}

// The part of n keys that this block of threads reads; parts: of how many, `most` at most. Parts begin
// at multiples of 64 keys.
__device__ __forceinline__ bool attn_part(const AttnArgs& a, int n, int split, int most, int& parts, int& from, int& to) {
  parts = min(max((n + a.chunk - 1) / a.chunk, 1), most);
  const int per = ((n + parts - 1) / parts + 63) & ~63;
  from = min(split * per, n);
  to = min(from + per, n);
  return split < parts;
}

// What a row's outputs are multiplied by at the end, and its log-sum-exp, from its maximum
// in base 2 and its sum (1 or more but for roundings, or 0). Only a sum of zero is a row that sees
// nothing: NaN stays NaN.
__device__ __forceinline__ float attn_inverse(float l) { return l == 0.0f ? 0.0f : 1.0f / l; }
__device__ __forceinline__ float attn_lse(float m, float l) { return l == 0.0f ? -INFINITY : (m + __builtin_amdgcn_logf(l)) * kLn2; }

__device__ __forceinline__ bool not_finite(float x) { return (__float_as_uint(x) & 0x7F800000u) == 0x7F800000u; }

}  // namespace rc
