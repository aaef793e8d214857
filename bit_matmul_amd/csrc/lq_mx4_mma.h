// Device helpers of the 4-bit products (mx4_gemm.hip, mx4_few.hip, mx4_token.hip).
#pragma once

#include "lq_int8.h"
#include "lq_mx4.h"

namespace lq {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

// acc + a c for 16 rows x 16 tokens x 128 values: lane (g, r) gives block g of
// its row, 32 codes, and in byte U of sa and sc that block's scales.
template <int U>
__device__ __forceinline__ f32x4 mfma_mx4(i32x4 a, i32x4 c, f32x4 acc, int sa, int sc) {
  const i32x8 a8 = {a[0], a[1], a[2], a[3], 0, 0, 0, 0}, c8 = {c[0], c[1], c[2], c[3], 0, 0, 0, 0};
  return __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a8, c8, acc, 4, 4, U, sa, U, sc);
}

// Of a block's 32 codes, as four dwords, those below `left`.
__device__ __forceinline__ uint32_t mx4_mask(int left, int i) {
  return left >= 8 * i + 8 ? 0xFFFFFFFFu : left <= 8 * i ? 0u : (1u << (4 * (left - 8 * i))) - 1u;
}
// Of a row's 8 scale bytes for 256 values, as two dwords, those of blocks below `left` (byte 2 g + s: block 4 s + g).
__device__ __forceinline__ uint32_t mx4_scale_mask(int left, int i) {
  uint32_t m = 0;
#pragma unroll
  for (int b = 0; b < 4; ++b) m |= 4 * (b & 1) + 2 * i + (b >> 1) < left ? 0xFFu << (8 * b) : 0u;
  return m;
}

// The scales and biases of rows n .. n + 3 (rows past N as the last one; none: 1
// and 0), all of them on their way at once.
__device__ __forceinline__ void load_mx4_rows(const Mx4Gemm& p, int64_t n, float (&rs)[4], float (&bias)[4]) {
#pragma unroll
  for (int e = 0; e < 4; ++e) rs[e] = 1.0f, bias[e] = 0.0f;
  if (p.row_scale != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) rs[e] = p.row_scale[min(n + e, p.N - 1)];
  }
  if (p.bias != nullptr) {
#pragma unroll
    for (int e = 0; e < 4; ++e) bias[e] = p.bias[min(n + e, p.N - 1)];
  }
}

// Outputs n .. n + 3 (those below N) of token b from their sums. Rows of y need
// only their element's alignment.
__device__ __forceinline__ void store_mx4_sums(const Mx4Gemm& p, int64_t b, int64_t n, const float (&rs)[4],
                                               const float (&bias)[4], f32x4 sum) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = fmaf(sum[e], rs[e], bias[e]);
  if (p.y_bf16) {
    uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + b * p.ldy + n;
    const uint32_t w[2] = {f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16),
                           f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16)};
    if (n + 4 <= p.N) __builtin_memcpy(y, w, 8);
    else
      for (int e = 0; e < 4 && n + e < p.N; ++e) y[e] = (uint16_t)(w[e >> 1] >> (16 * (e & 1)));
  } else {
    float* y = reinterpret_cast<float*>(p.y) + b * p.ldy + n;
    if (n + 4 <= p.N) __builtin_memcpy(y, v, 16);
    else
      for (int e = 0; e < 4 && n + e < p.N; ++e) y[e] = v[e];
  }
}

}  // namespace lq
