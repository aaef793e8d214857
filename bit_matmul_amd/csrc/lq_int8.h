// Device helpers of the 8-bit products (int8_gemm.hip, int8_few.hip,
// int8_token.hip).
#pragma once

#include "lq_8bit.h"

namespace lq {

typedef __attribute__((ext_vector_type(4))) int i32x4;

// A barrier for LDS alone (__syncthreads would wait for the copies in flight):
// this wavefront's accesses are done before it. The builtins say nothing to
// the compiler about memory: the fences, which are no instructions, keep
// accesses on their side of it.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_s_waitcnt(3 << 14 | 7 << 4 | 15);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
}

// Outputs n .. n + 3 (those below N) of token b from their sums, with the
// token's scale sb, the rows' scales rs and biases. Rows of y need only
// their element's alignment.
__device__ __forceinline__ void store_int8_sums(const Int8Gemm& p, int64_t b, int64_t n, float sb,
                                                const float (&rs)[4], const float (&bias)[4], i32x4 sum) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) v[e] = fmaf((float)sum[e], sb * rs[e], bias[e]);
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

// The scales and biases of rows n .. n + 3 (rows past N as the last one).
__device__ __forceinline__ void load_int8_rows(const Int8Gemm& p, int64_t n, float (&rs)[4], float (&bias)[4]) {
  if (n + 4 <= p.N) {
    __builtin_memcpy(rs, p.row_scale + n, 16);
  } else {
#pragma unroll
    for (int e = 0; e < 4; ++e) rs[e] = p.row_scale[min(n + e, p.N - 1)];
  }
#pragma unroll
  for (int e = 0; e < 4; ++e) bias[e] = 0.0f;
  if (p.bias != nullptr) {
    if (n + 4 <= p.N) {
      __builtin_memcpy(bias, p.bias + n, 16);
    } else {
#pragma unroll
      for (int e = 0; e < 4; ++e) bias[e] = p.bias[min(n + e, p.N - 1)];
    }
  }
}

}  // namespace lq
