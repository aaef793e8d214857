// Device helpers of the 8-bit products (int8_stream.hip, int8_tile.hip).
#pragma once

#include "lq_internal.h"

namespace lq {

typedef __attribute__((ext_vector_type(4))) int i32x4;

// Outputs n .. n + 3 (those below N) of token b from their sums; sb is the
// token's scale. Rows of y need only their element's alignment.
__device__ __forceinline__ void store_int8_sums(const Int8Gemm& p, int64_t b, int64_t n, float sb,
                                                i32x4 sum) {
  float v[4];
  if (n + 4 <= p.N) {
    float rs[4], bias[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    __builtin_memcpy(rs, p.row_scale + n, 16);
    if (p.bias != nullptr) __builtin_memcpy(bias, p.bias + n, 16);
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = fmaf((float)sum[e], sb * rs[e], bias[e]);
    if (p.y_bf16) {
      const uint32_t w[2] = {f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16),
                             f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16)};
      __builtin_memcpy(reinterpret_cast<uint16_t*>(p.y) + b * p.ldy + n, w, 8);
    } else {
      __builtin_memcpy(reinterpret_cast<float*>(p.y) + b * p.ldy + n, v, 16);
    }
    return;
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    if (n + e >= p.N) break;
    const float o = fmaf((float)sum[e], sb * p.row_scale[n + e], p.bias != nullptr ? p.bias[n + e] : 0.0f);
    if (p.y_bf16) reinterpret_cast<uint16_t*>(p.y)[b * p.ldy + n + e] = (uint16_t)f32_to_bf16_bits(o);
    else reinterpret_cast<float*>(p.y)[b * p.ldy + n + e] = o;
  }
}

}  // namespace lq
