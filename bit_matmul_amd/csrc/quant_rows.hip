// 8-bit rows: v = T (act(gate) .* x), s = max|v| / 127, q = v 127 / max|v|
// rounded to the nearest whole number (ties to even): the activations of the
// 8-bit product. act(gate) and T (the lifted layer's channel scales and block
// Hadamard transform) are each optional.
//
// One workgroup per row, the row in registers (lq_rows.h): it is read once,
// its maximum is one reduction over the workgroup, and the codes are written
// from the same registers. Without T the time is that of the bytes. Replays of
// a graph, so that a launch's 3 to 4 us between kernels are in the times, rows
// from memory: 2048 rows of 8192 in bf16 16 us (3.1 TB/s; the kernel alone, its
// rows in the cache, 12.4), of 28672 44 (4.0 TB/s), gated 67 (4.4); in fp32 56
// (5.3 TB/s), gated 130 (4.1). One row of 8192 3.4 us.
//
// With T it is not: every row's workgroup reads the channel scales too, which
// are twice a bf16 row, and 10 butterflies a value stand beside it: 8192 19 us,
// 28672 66 (2.7 TB/s), gated 115, fp32 85 and gated 189.
//
// Registers do not hold everything: of the rows of 16385 to 32768 values (C 2)
// the fp32 forms with a gate spill (44 bytes of scratch a lane, with T 76), the
// bf16 form with T a little (12), and the fp32 form with T and without a gate
// keeps its scales in 41 KB of LDS; past 32768 (C 4) the fp32 form with a gate
// spills 60 bytes: 256 rows of 40000 32 us (2.9 TB/s), plain bf16 17 (1.9).
#include <type_traits>

#include "lq_rows.h"

namespace lq {
namespace {

// Wavefronts on a SIMD: without T two workgroups' registers have room (gated
// rows of 28672), so that one loads while the other computes. With T (kT) the
// channel scales are loaded along with the row instead: few rows wait for
// memory once, not twice.
template <int C, bool kXBF16, bool kGate, bool kT>
__global__ __launch_bounds__(1024, (C == 4 ? 4 : kT ? 5 : C == 2 ? 7 : 8)) void quant_rows_kernel(QuantRows p) {
  __shared__ float red[kRowMaxWaves];
  const int64_t b = blockIdx.x;
  const int K = (int)p.K;
  const bool whole = row_whole<C>(K);
  const char* const xrow = reinterpret_cast<const char*>(p.x) + b * p.ldx * (kXBF16 ? 2 : 4);
  const char* const grow = reinterpret_cast<const char*>(p.gate) + b * p.ldg * (kXBF16 ? 2 : 4);
  float v[C][2][8];
  float m = 0.0f;
  // G blocks' loads at a time
  constexpr int G = C == 4 ? 1 : C;
#pragma unroll
  for (int i0 = 0; i0 < C; i0 += G) {
    RowPiece<kXBF16> x[G][2], g[G][2];
    RowPiece<false> c[G][2];
    auto load = [&](auto wholec) __attribute__((always_inline)) {
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          load_piece(x[i][j], xrow, row_col(i0 + i, j), K, decltype(wholec)::value);
          if constexpr (kGate) load_piece(g[i][j], grow, row_col(i0 + i, j), K, decltype(wholec)::value);
        }
      if (kT && p.c != nullptr) {
#pragma unroll
        for (int i = 0; i < G; ++i)
#pragma unroll
          for (int j = 0; j < 2; ++j) load_piece(c[i][j], p.c, row_col(i0 + i, j), K, decltype(wholec)::value);
      }
    };
    if (whole) load(std::true_type{});
    else load(std::false_type{});
#pragma unroll
    for (int i = 0; i < G; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float a[8];
        x[i][j].get(v[i0 + i][j]);
        if constexpr (kGate) {
          g[i][j].get(a);
          act_row8(p.act, a);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i0 + i][j][k] *= a[k];
        }
      }
    if (kT && p.c != nullptr) {
#pragma unroll
      for (int i = 0; i < G; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float a[8];
          c[i][j].get(a);
#pragma unroll
          for (int k = 0; k < 8; ++k) v[i0 + i][j][k] *= a[k];
        }
    }
    if constexpr (C == 4) __builtin_amdgcn_sched_barrier(0);
  }
  if (kT && p.lhb > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) fwht_block(v[i], p.lhb);
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(v[i][j][k]));
  m = row_reduce<MaxBits>(m, red);
  // (the transform's 1 / sqrt(hb) scales v and its maximum alike: the codes
  // do not see it)
  const RowCoder coder(m);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    uint2 w[2] = {coder.codes(v[i][0]), coder.codes(v[i][1])};
    if (kT && p.lhb > 7) fwht_order(w, p.lhb);
#pragma unroll
    for (int j = 0; j < 2; ++j) store_codes(p.q + b * p.ldq, row_col(i, j), K, w[j]);
  }
  if (threadIdx.x == 0) p.scale[b] = coder.scale(p.norm);
}

template <int C, bool kT>
void enqueue(const QuantRows& p, dim3 grid, dim3 block, hipStream_t stream) {
  if (p.x_bf16) {
    if (p.gate) hipLaunchKernelGGL((quant_rows_kernel<C, true, true, kT>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((quant_rows_kernel<C, true, false, kT>), grid, block, 0, stream, p);
  } else {
    if (p.gate) hipLaunchKernelGGL((quant_rows_kernel<C, false, true, kT>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((quant_rows_kernel<C, false, false, kT>), grid, block, 0, stream, p);
  }
}
template <int C>
void enqueue(const QuantRows& p, dim3 grid, dim3 block, hipStream_t stream) {
  if (p.c != nullptr || p.lhb > 0) enqueue<C, true>(p, grid, block, stream);
  else enqueue<C, false>(p, grid, block, stream);
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
