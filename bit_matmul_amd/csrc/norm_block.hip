// The norms around a block with its gate and scaled residual, one row per
// workgroup (include/lq.h gives the formulas):
//
//   u  = y (.* act(gate))            gate first
//   u  = u / rms(u) .* w_post        norm after the block
//   u  = u (.* act(gate))            gate last
//   h' = h + alpha u
//   a  = h' / rms(h') .* w_pre       norm before the next block, as values
//                                    or as 8-bit codes with a scale
//
// Read once, kept in registers (lq_rows.h), written once: the time is that of
// the bytes. The second norm reads h' as it was summed in 32 bits, before it
// is rounded to the residual stream's type. Squares are summed in 32 bits,
// each thread its 16 C values, then a butterfly over lanes and wavefronts.
#include "lq_rows.h"

namespace lq {
namespace {

// 1 / sqrt(mean(v^2) + eps). Where the sum of squares passes the largest
// float, v becomes v 2^-80 and the sum is taken again (every thread of the
// workgroup sees the same sum, so all take the branch together): eps is
// nothing there, and the norm of v does not change.
template <int C>
__device__ __forceinline__ float inv_rms(float (&v)[C][2][8], int K, float eps, float* red) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) s = fmaf(v[i][j][k], v[i][j][k], s);
  s = row_reduce<SumF>(s, red);
  if (s <= 3.0e38f) return 1.0f / sqrtf(s / (float)K + eps);
  s = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][j][k] *= 0x1p-80f;
        s = fmaf(v[i][j][k], v[i][j][k], s);
      }
  s = row_reduce<SumF>(s, red + kRowMaxWaves);
  return 1.0f / sqrtf(s / (float)K);
}

template <int C>
__device__ __forceinline__ void apply_norm(float (&v)[C][2][8], float r, const float* w, bool one_plus,
                                           int K, int wave, int waves, int lane) {
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int s = (wave + i * waves) * kRowBlock + 512 * j + 8 * lane;
      float g[8];
      if (w != nullptr) load_row8<false>(w, s, K - s, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float wk = w == nullptr ? 1.0f : one_plus ? 1.0f + g[k] : g[k];
        v[i][j][k] = v[i][j][k] * r * wk;
      }
    }
}

template <int C, bool kYBF16, bool kHBF16>
__global__ __launch_bounds__(1024) void norm_block_kernel(NormBlock p) {
  __shared__ float red[5][kRowMaxWaves];
  const int wave = wave_id(), lane = threadIdx.x & 63, waves = (int)blockDim.x >> 6;
  const int64_t b = blockIdx.x;
  const int K = (int)p.K;
  float v[C][2][8];
  auto each = [&](auto fn) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) fn(v[i][j], (wave + i * waves) * kRowBlock + 512 * j + 8 * lane);
  };
  auto gate = [&] __attribute__((always_inline)) {
    each([&](float (&u)[8], int s) __attribute__((always_inline)) {
      float g[8];
      load_row8<kYBF16>(p.gate, b * p.ldg + s, K - s, g);
      act_row8(p.act, g);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] *= g[k];
    });
  };
  if (p.y != nullptr) {
    each([&](float (&u)[8], int s) __attribute__((always_inline)) {
      load_row8<kYBF16>(p.y, b * p.ldy + s, K - s, u);
    });
    if (p.gate != nullptr && p.gate_first) gate();
    if (p.post)
      apply_norm<C>(v, inv_rms<C>(v, K, p.eps, red[0]), p.w_post, p.one_plus, K, wave, waves, lane);
    if (p.gate != nullptr && !p.gate_first) gate();
  }
  if (p.h != nullptr) {
    each([&](float (&u)[8], int s) __attribute__((always_inline)) {
      float h[8];
      load_row8<kHBF16>(p.h, b * p.ldh + s, K - s, h);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = p.y != nullptr ? fmaf(p.alpha, u[k], h[k]) : h[k];
    });
  } else {
    each([&](float (&u)[8], int) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] *= p.alpha;
    });
  }
  if (p.h_out != nullptr)
    each([&](float (&u)[8], int s) __attribute__((always_inline)) {
      store_row8(p.h_out, kHBF16, b * p.ldho + s, K - s, u);
    });
  if (p.pre)
    apply_norm<C>(v, inv_rms<C>(v, K, p.eps, red[2]), p.w_pre, p.one_plus, K, wave, waves, lane);
  if (p.a != nullptr)
    each([&](float (&u)[8], int s) __attribute__((always_inline)) {
      store_row8(p.a, p.a_bf16, b * p.lda + s, K - s, u);
    });
  if (p.q != nullptr) {
    float m = 0.0f;
    each([&](float (&u)[8], int) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(u[k]));
    });
    m = row_reduce<MaxBits>(m, red[4]);
    const RowCoder coder(m);
    each([&](float (&u)[8], int s) __attribute__((always_inline)) {
      store_codes(p.q, b * p.ldq, s, K, coder.codes(u));
    });
    if (threadIdx.x == 0) p.scale[b] = coder.scale(m);
  }
}

template <int C>
void enqueue(const NormBlock& p, dim3 grid, dim3 block, hipStream_t stream) {
  if (p.y_bf16) {
    if (p.h_bf16) hipLaunchKernelGGL((norm_block_kernel<C, true, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((norm_block_kernel<C, true, false>), grid, block, 0, stream, p);
  } else {
    if (p.h_bf16) hipLaunchKernelGGL((norm_block_kernel<C, false, true>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((norm_block_kernel<C, false, false>), grid, block, 0, stream, p);
  }
}

}  // namespace

hipError_t launch_norm_block(const NormBlock& p, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const RowShape s = row_shape(p.K);
  const dim3 grid((unsigned)p.B), block(64u * (unsigned)s.waves);
  if (s.c == 1) enqueue<1>(p, grid, block, stream);
  else if (s.c == 2) enqueue<2>(p, grid, block, stream);
  else enqueue<4>(p, grid, block, stream);
  return hipGetLastError();
}

}  // namespace lq
