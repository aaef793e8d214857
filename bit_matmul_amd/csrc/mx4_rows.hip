// Microscaled 4-bit rows (include/lq.h gives the format) of v = T (act(gate)
// .* x): the rows and weights of the 4-bit product.
//
// A block's scale needs its own 32 values alone, T its own 1024, so no
// wavefront waits for another: each takes 1024 values of a row (lq_rows.h:
// a lane 8 values of each half), a block is four lanes, and its maximum two
// lane exchanges. The conversion is the hardware's: v_cvt_scalef32_pk_fp4_f32
// divides by the power of two, which is exact, and rounds to the nearest value,
// ties to the even code, what is above 6 to 6.
#include <type_traits>

#include "lq_mx4.h"
#include "lq_rows.h"

namespace lq {
namespace {

// Undoes what fwht_block's exchanges of lane and register bits did to the
// places of values: afterwards v is in the order of its columns again.
__device__ __forceinline__ void fwht_restore(float (&v)[2][8], int lhb) {
  auto swap = [&](auto bit, float& a, float& b) __attribute__((always_inline)) {
    uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    lane_swap<decltype(bit)::value>(x, y);
    a = __uint_as_float(x);
    b = __uint_as_float(y);
  };
  if (lhb > 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) swap(std::integral_constant<int, 32>{}, v[0][k], v[1][k]);
  }
  if (lhb > 7) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) swap(std::integral_constant<int, 16>{}, v[j][k], v[j][k + 4]);
  }
}

// The scale byte of a block whose largest magnitude has these bits.
__device__ __forceinline__ uint32_t mx4_scale_byte(uint32_t bits) {
  const uint32_t e = bits >> 23;
  return e == 255u ? 255u : e > 2u ? e - 2u : 0u;
}

// 8 codes, the first in the lowest bits, of v 2^(127 - byte).
__device__ __forceinline__ uint32_t mx4_codes(const float (&v)[8], uint32_t byte) {
  // (2^-127 lies below the normal floats)
  const float scale = __uint_as_float(byte > 0u ? byte << 23 : 0x400000u);
  uint32_t o = 0;
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[0], v[1], scale, 0);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[2], v[3], scale, 1);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[4], v[5], scale, 2);
  o = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(o, v[6], v[7], scale, 3);
  return byte == 255u ? 0u : o;
}

template <bool kXBF16, bool kGate, bool kT>
__global__ __launch_bounds__(256) void mx4_rows_kernel(Mx4Rows p) {
  const int64_t b = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  const int K = (int)p.K;
  const int col0 = ((int)blockIdx.y * ((int)blockDim.x >> 6) + wave_id()) * kRowBlock;
  if (b >= p.B || col0 >= K) return;
  const int lane = threadIdx.x & 63;
  const bool whole = col0 + kRowBlock <= K;
  const char* const xrow = reinterpret_cast<const char*>(p.x) + b * p.ldx * (kXBF16 ? 2 : 4);
  const char* const grow = reinterpret_cast<const char*>(p.gate) + b * p.ldg * (kXBF16 ? 2 : 4);
  RowPiece<kXBF16> x[2], g[2];
  RowPiece<false> c[2];
  float v[2][8];
  auto load = [&](auto wholec) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      load_piece(x[j], xrow, col0 + 512 * j, K, decltype(wholec)::value);
      if constexpr (kGate) load_piece(g[j], grow, col0 + 512 * j, K, decltype(wholec)::value);
    }
    if (kT && p.c != nullptr) {
#pragma unroll
      for (int j = 0; j < 2; ++j) load_piece(c[j], p.c, col0 + 512 * j, K, decltype(wholec)::value);
    }
  };
  if (whole) load(std::true_type{});
  else load(std::false_type{});
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    x[j].get(v[j]);
    if constexpr (kGate) {
      float a[8];
      g[j].get(a);
      act_row8(p.act, a);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= a[k];
    }
    if (kT && p.c != nullptr) {
      float a[8];
      c[j].get(a);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= a[k];
    }
  }
  if (kT && p.lhb > 0) {
    fwht_block(v, p.lhb);
    fwht_restore(v, p.lhb);
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= p.norm;
  }
  const int units = (int)mx4_units(p.K), bytes = (int)mx4_row_bytes(p.K);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    float m = 0.0f;
#pragma unroll
    for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(v[j][k]));
    m = MaxBits::of(m, lane_xor<1>(m));
    m = MaxBits::of(m, lane_xor<2>(m));
    const uint32_t byte = mx4_scale_byte(__float_as_uint(m));
    const int at = (col0 + 512 * j) / 2 + 4 * lane;
    if (at < bytes) *reinterpret_cast<uint32_t*>(p.q + b * p.ldq + at) = mx4_codes(v[j], byte);
    // the first lane of a block: block i of unit u
    const int u = (col0 + 512 * j) / kMxUnit + (lane >> 5), i = (lane >> 2) & 7;
    if ((lane & 3) == 0 && u < units)
      p.scale[((b >> 4) * units + u) * 128 + 8 * (b & 15) + 2 * (i & 3) + (i >> 2)] = (uint8_t)byte;
  }
}

constexpr int64_t kGridRows = 1 << 22;

template <bool kT>
void enqueue(const Mx4Rows& p, dim3 grid, dim3 block, hipStream_t stream) {
  if (p.x_bf16) {
    if (p.gate) hipLaunchKernelGGL((mx4_rows_kernel<true, true, kT>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((mx4_rows_kernel<true, false, kT>), grid, block, 0, stream, p);
  } else {
    if (p.gate) hipLaunchKernelGGL((mx4_rows_kernel<false, true, kT>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((mx4_rows_kernel<false, false, kT>), grid, block, 0, stream, p);
  }
}

}  // namespace

hipError_t launch_mx4_rows(const Mx4Rows& p, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const int blocks = (int)((p.K + kRowBlock - 1) / kRowBlock), waves = blocks < 4 ? blocks : 4;
  // (a launch has fewer than 2^32 threads along an axis)
  const int64_t rows = p.B < kGridRows ? p.B : kGridRows;
  const dim3 grid((unsigned)rows, (unsigned)((blocks + waves - 1) / waves), (unsigned)((p.B + rows - 1) / rows));
  const dim3 block(64u * (unsigned)waves);
  if (p.c != nullptr || p.lhb > 0) enqueue<true>(p, grid, block, stream);
  else enqueue<false>(p, grid, block, stream);
  return hipGetLastError();
}

}  // namespace lq
