// 8-bit rows: v = T (act(gate) .* x), s = max|v| / 127, q = v 127 / max|v|
// rounded to the nearest whole number (ties to even): the activations of the
// 8-bit product. act(gate) and T (the lifted layer's channel scales and block
// Hadamard transform) are each optional.
//
// One workgroup per row, the row in registers (lq_rows.h): it is read once,
// its maximum is one reduction over the workgroup, and the codes are written
// from the same registers. The time is that of the bytes.
#include "lq_rows.h"

namespace lq {
namespace {

// Stage `bit` of the transform is a butterfly over bit `bit` of the index
// within the block: bits 0..2 pair the 8 values of a piece, bits 3..8 pair
// lanes, bit 9 pairs the two pieces.
__device__ __forceinline__ void fwht_block(float (&v)[2][8], int lhb, int lane) {
  float a[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) a[k] = v[k >> 3][k & 7];
#pragma unroll
  for (int s = 0; s < 3; ++s)
    if (s < lhb) {
#pragma unroll
      for (int k = 0; k < 16; ++k)
        if ((k & (1 << s)) == 0) {
          const float x0 = a[k], x1 = a[k | (1 << s)];
          a[k] = x0 + x1;
          a[k | (1 << s)] = x0 - x1;
        }
    }
  if (lhb > 3) lane_stage<1>(a, lane);
  if (lhb > 4) lane_stage<2>(a, lane);
  if (lhb > 5) lane_stage<4>(a, lane);
  if (lhb > 6) lane_stage<8>(a, lane);
  if (lhb > 7) lane_stage<16>(a, lane);
  if (lhb > 8) lane_stage<32>(a, lane);
  if (lhb > 9) {
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const float x0 = a[k], x1 = a[k + 8];
      a[k] = x0 + x1;
      a[k + 8] = x0 - x1;
    }
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k >> 3][k & 7] = a[k];
}

template <int C, bool kXBF16, bool kGate>
__global__ __launch_bounds__(1024) void quant_rows_kernel(QuantRows p) {
  __shared__ float red[kRowMaxWaves];
  const int wave = wave_id(), lane = threadIdx.x & 63, waves = (int)blockDim.x >> 6;
  const int64_t b = blockIdx.x;
  float v[C][2][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int s = (wave + i * waves) * kRowBlock + 512 * j + 8 * lane;
      load_row8<kXBF16>(p.x, b * p.ldx + s, (int)p.K - s, v[i][j]);
    }
  }
  if constexpr (kGate) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int s = (wave + i * waves) * kRowBlock + 512 * j + 8 * lane;
        float g[8];
        load_row8<kXBF16>(p.gate, b * p.ldg + s, (int)p.K - s, g);
        act_row8(p.act, g);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][j][k] *= g[k];
      }
    }
  }
  if (p.c != nullptr) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const int s = (wave + i * waves) * kRowBlock + 512 * j + 8 * lane;
        float c[8];
        load_row8<false>(p.c, s, (int)p.K - s, c);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][j][k] *= c[k];
      }
    }
  }
  if (p.lhb > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      fwht_block(v[i], p.lhb, lane);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][j][k] *= p.norm;
    }
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(v[i][j][k]));
  m = row_reduce<MaxBits>(m, red);
  const RowCoder coder(m);
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int s = (wave + i * waves) * kRowBlock + 512 * j + 8 * lane;
      store_codes(p.q, b * p.ldq, s, p.K, coder.codes(v[i][j]));
    }
  if (threadIdx.x == 0) p.scale[b] = coder.scale(m);
}

template <int C>
void enqueue(const QuantRows& p, dim3 grid, dim3 block, hipStream_t stream) {
  if (p.x_bf16) {
    if (p.gate) hipLaunchKernelGGL((quant_rows_kernel<C, true, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((quant_rows_kernel<C, true, false>), grid, block, 0, stream, p);
  } else {
    if (p.gate) hipLaunchKernelGGL((quant_rows_kernel<C, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((quant_rows_kernel<C, false, false>), grid, block, 0, stream, p);
  }
}

}  // namespace

RowShape row_shape(int64_t K) {
  const int blocks = (int)((K + kRowBlock - 1) / kRowBlock);
  const int c = blocks <= kRowMaxWaves ? 1 : blocks <= 2 * kRowMaxWaves ? 2 : 4;
  return {c, (blocks + c - 1) / c};
}

hipError_t launch_quant_rows(const QuantRows& p, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const RowShape s = row_shape(p.K);
  const dim3 grid((unsigned)p.B), block(64u * (unsigned)s.waves);
  if (s.c == 1) enqueue<1>(p, grid, block, stream);
  else if (s.c == 2) enqueue<2>(p, grid, block, stream);
  else enqueue<4>(p, grid, block, stream);
  return hipGetLastError();
}

}  // namespace lq
