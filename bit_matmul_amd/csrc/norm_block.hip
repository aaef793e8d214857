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
// each thread its 16 C values in four chains (one chain of them may lose 15
// roundings where its first value is the large one), then a butterfly over
// lanes and wavefronts.
//
// Measured in replays of a graph, tensors from memory (in brackets: the same
// ones again, from the cache): 2048 rows of 8192 in bf16, both norms and 8-bit
// rows 30 us (26; 3.9 and 4.6 TB/s), in fp32 without 8-bit rows 53 (43; 5.1 and
// 6.3); 777 rows of 4099 in fp32 with a gate 20 (16; 3.3 and 4.0); one row 3.8
// to 5.2 us (the launch, memory, two reductions). Rows past 32768 (C = 4) spill
// 84 to 92 bytes of scratch a lane: 256 of 40000 37 us (31; 2.2 and 2.6).
#include "lq_rows.h"

namespace lq {
namespace {

// The sum of (f(v))^2 over a thread's values: chain k & 3, joined pairwise.
template <int C, typename F>
__device__ __forceinline__ float sum_squares(float (&v)[C][2][8], F f) {
  float s[4] = {};
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        const float w = f(v[i][j][k]);
        s[k & 3] = fmaf(w, w, s[k & 3]);
      }
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// 1 / sqrt(mean(v^2) + eps). Where the sum of squares, or the mean's with a large
// eps, passes the largest float, it is taken again of v 2^-80 (every thread of the workgroup sees the
// same sum, so all take the branch together), with eps 2^-160 (0 below 2^11,
// which is nothing next to a mean of 4.6e33 or more). The root is then 2^80
// times too large, and half of that factor goes into v: the norm stays what it
// is, and neither the root nor a v whose norm is a normal float (8e-22 or more)
// leaves the normal floats.
template <int C>
__device__ __forceinline__ float inv_rms(float (&v)[C][2][8], int K, float eps, float* red) {
  float s = row_reduce<SumF>(sum_squares<C>(v, [](float& u) { return u; }), red);
  const float mean = s / (float)K + eps;
  if (s <= 3.0e38f && mean <= 3.4e38f) return inv_root(mean);
  s = row_reduce<SumF>(sum_squares<C>(v, [](float& u) { return (u *= 0x1p-40f) * 0x1p-40f; }),
                       red + kRowMaxWaves);
  return inv_root(s / (float)K + eps * 0x1p-80f * 0x1p-80f) * 0x1p-40f;
}

// Each tensor is loaded where it is first used. All loads before the first
// reduction, which the registers of one block of 1024 have room for, gave
// nothing for few rows (64 rows of 8192 with both norms 5.8 -> 6.0 us) and
// cost many (2048 rows 26.9 -> 30.0 us: fewer workgroups fit).
template <int C, bool kYBF16, bool kHBF16>
__global__ __launch_bounds__(1024, (C == 1 ? 8 : 4)) void norm_block_kernel(NormBlock p) {
  __shared__ float red[5][kRowMaxWaves];
  const int64_t b = blockIdx.x;
  const int K = (int)p.K;
  const bool whole = C < 4 && row_whole<C>(K);
  float v[C][2][8];
  RowPiece<kYBF16> y[2], g[2];
  RowPiece<kHBF16> h[2];
  auto row = [&](const void* base, int64_t ld, bool bf16) __attribute__((always_inline)) {
    return reinterpret_cast<const char*>(base) + b * ld * (bf16 ? 2 : 4);
  };
  // the pieces of block i of a row
  auto load = [&](auto& piece, const void* from, int i) __attribute__((always_inline)) {
    if (whole) {
#pragma unroll
      for (int j = 0; j < 2; ++j) load_piece(piece[j], from, row_col(i, j), K, true);
    } else {
#pragma unroll
      for (int j = 0; j < 2; ++j) load_piece(piece[j], from, row_col(i, j), K, false);
    }
  };
  const char* const yrow = row(p.y, p.ldy, kYBF16);
  const char* const grow = row(p.gate, p.ldg, kYBF16);
  const char* const hrow = row(p.h, p.ldh, kHBF16);
  auto load_weights = [&](RowPiece<false> (&piece)[2], const float* w, int i) __attribute__((always_inline)) {
    if (w != nullptr) load(piece, w, i);
  };
  // fn(values, block, piece) for all of a thread's pieces
  auto each = [&](auto fn) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) fn(v[i][j], i, j);
      if constexpr (C == 4) __builtin_amdgcn_sched_barrier(0);   // (one block's loads in registers at a time)
    }
  };
  auto gate = [&] __attribute__((always_inline)) {
    each([&](float (&u)[8], int i, int j) __attribute__((always_inline)) {
      if (j == 0) load(g, grow, i);
      float a[8];
      g[j].get(a);
      act_row8(p.act, a);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] *= a[k];
    });
  };
  auto norm = [&](float* lds, const float* w) __attribute__((always_inline)) {
    RowPiece<false> wp[2];
    const float r = inv_rms<C>(v, K, p.eps, lds);
    const float plus = p.one_plus ? 1.0f : 0.0f;
    each([&](float (&u)[8], int i, int j) __attribute__((always_inline)) {
      if (j == 0) load_weights(wp, w, i);
      float a[8];
      wp[j].get(a);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = u[k] * r * (w != nullptr ? plus + a[k] : 1.0f);
    });
  };
  if (p.y != nullptr) {
    each([&](float (&u)[8], int i, int j) __attribute__((always_inline)) {
      if (j == 0) load(y, yrow, i);
      y[j].get(u);
    });
    if (p.gate != nullptr && p.gate_first) gate();
    if (p.post) norm(red[0], p.w_post);
    if (p.gate != nullptr && !p.gate_first) gate();
  }
  if (p.h != nullptr) {
    each([&](float (&u)[8], int i, int j) __attribute__((always_inline)) {
      if (j == 0) load(h, hrow, i);
      float a[8];
      h[j].get(a);
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] = p.y != nullptr ? fmaf(p.alpha, u[k], a[k]) : a[k];
    });
  } else {
    each([&](float (&u)[8], int, int) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) u[k] *= p.alpha;
    });
  }
  if (p.h_out != nullptr)
    each([&](float (&u)[8], int i, int j) __attribute__((always_inline)) {
      store_row8(const_cast<char*>(row(p.h_out, p.ldho, kHBF16)), kHBF16, row_col(i, j), K, whole, u);
    });
  if (p.pre) norm(red[2], p.w_pre);
  if (p.a != nullptr)
    each([&](float (&u)[8], int i, int j) __attribute__((always_inline)) {
      store_row8(const_cast<char*>(row(p.a, p.lda, p.a_bf16)), p.a_bf16, row_col(i, j), K, whole, u);
    });
  if (p.q != nullptr) {
    float m = 0.0f;
    each([&](float (&u)[8], int, int) __attribute__((always_inline)) {
#pragma unroll
      for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(u[k]));
    });
    m = row_reduce<MaxBits>(m, red[4]);
    const RowCoder coder(m);
    each([&](float (&u)[8], int i, int j) __attribute__((always_inline)) {
      store_codes(p.q + b * p.ldq, row_col(i, j), K, coder.codes(u));
    });
    if (threadIdx.x == 0) p.scale[b] = coder.scale(1.0f);
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
