// Device helpers of the key/value cache kernels.
#pragma once

#include "device_common.hpp"
#include "kv.hpp"

namespace rc {

typedef _Float16 half2_t __attribute__((ext_vector_type(2)));
typedef _Float16 half8_t __attribute__((ext_vector_type(8)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));
typedef int i32x16 __attribute__((ext_vector_type(16)));

// Pool index of block j of sequence b, or -1 where there is none.
__device__ __forceinline__ int kv_block(const KvGeom& g, int b, int j) {
  const int p = g.table ? g.table[(int64_t)b * g.seq_blocks + j] : b * g.seq_blocks + j;
  return (unsigned)p < (unsigned)g.pool_blocks ? p : -1;
}
// Index of the (block, key head) row that scales and means have.
__device__ __forceinline__ int64_t kv_row(const KvGeom& g, int block, int head) {
  return (int64_t)block * g.kv_heads + head;
}

__device__ __forceinline__ int kv_length(const KvAttendArgs& a, int b) {
  return min(max(a.kv_len[b], 0), a.max_len);
}
// Tokens that query i sees.
__device__ __forceinline__ int kv_limit(const KvAttendArgs& a, int len, int i) {
  return a.causal ? max(0, len - a.queries + i + 1) : len;
}

__device__ __forceinline__ float pow2f(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }
// Exponent of a power of two that the cache holds, kept in the allowed range
// whatever the memory holds.
__device__ __forceinline__ int scale_exponent(float s) {
  return min(max((int)(__float_as_uint(s) >> 23 & 255) - 127, kKvEMin), kKvEMax);
}

// 8 consecutive values of a row, as fp32.
template <typename IN>
__device__ __forceinline__ void row8(const IN* p, float (&x)[8]) {
  F8 t;
  load8<IN>(p, t);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = t.v[i];
}

// Two outputs as bf16, rounded to nearest even; a NaN of any payload stays one (bf16_rne is
// for finite values, and would carry a full payload into the sign).
typedef float f32x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
  return __builtin_bit_cast(uint32_t, __builtin_convertvector((f32x2{lo, hi}), bf16x2));
}

// Four e4m3 codes -> four f16 (exact: every e4m3 value is a normal f16).
__device__ __forceinline__ void codes4(uint32_t c, half2_t& lo, half2_t& hi) {
  lo = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, false);
  hi = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(c, 1.0f, true);
}
__device__ __forceinline__ half8_t codes8(uint32_t a, uint32_t b) {
  half2_t w, x, y, z;
  codes4(a, w, x);
  codes4(b, y, z);
  return half8_t{w.x, w.y, x.x, x.y, y.x, y.y, z.x, z.y};
}

}  // namespace rc
