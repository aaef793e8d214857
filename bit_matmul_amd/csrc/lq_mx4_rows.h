// Device helpers that make microscaled 4-bit rows (mx4_rows.hip,
// mx4_token.hip).
#pragma once

#include <type_traits>

#include "lq_mx4.h"
#include "lq_rows.h"

namespace lq {

// Undoes what fwht_stages' exchanges of lane and register bits did to the
// places of values: afterwards v is in the order of its columns again.
template <int kLaneBit>
__device__ __forceinline__ void swap_back(float& a, float& b) {
  uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
  lane_swap<kLaneBit>(x, y);
  a = __uint_as_float(x);
  b = __uint_as_float(y);
}
__device__ __forceinline__ void fwht_restore(float (&v)[2][8], int lhb) {
  if (lhb > 8) {
#pragma unroll
    for (int k = 0; k < 8; ++k) swap_back<32>(v[0][k], v[1][k]);
  }
  if (lhb > 7) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) swap_back<16>(v[j][k], v[j][k + 4]);
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

// A lane's 8 values of a piece of 512: their codes, and in `byte` the scale of
// their block, which four lanes share.
__device__ __forceinline__ uint32_t mx4_piece(const float (&v)[8], uint32_t& byte) {
  float m = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(v[k]));
  m = MaxBits::of(m, lane_xor<1>(m));
  m = MaxBits::of(m, lane_xor<2>(m));
  byte = mx4_scale_byte(__float_as_uint(m));
  return mx4_codes(v, byte);
}

// A piece of 8 values at column col of a row of K, a multiple of 8: of one past
// the row the row's last, which the caller drops (no branch, so that loads and
// what follows them are on their way at once).
template <bool kBF16>
__device__ __forceinline__ void load_even(RowPiece<kBF16>& p, const void* row, int col, int K) {
  const uint32_t at = (uint32_t)min(col + (int)row_lane8(), K - 8) * (kBF16 ? 2u : 4u);
  __builtin_memcpy(p.w, reinterpret_cast<const char*>(row) + at, sizeof(p.w));
}

// The pieces of a wavefront's 1024 values from column col0 on, as they lie in
// memory, and act(gate) .* x .* c of them. kEven: K is a multiple of 8.
template <bool kXBF16, bool kGate, bool kScaled, bool kEven>
struct Mx4Block {
  RowPiece<kXBF16> x[2], g[kGate ? 2 : 1];
  RowPiece<false> c[kScaled ? 2 : 1];
  __device__ __forceinline__ void load(const Mx4Rows& p, const char* xrow, const char* grow, int col0) {
    const int K = (int)p.K;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      if constexpr (kEven) {
        load_even(x[j], xrow, col0 + 512 * j, K);
        if constexpr (kGate) load_even(g[j], grow, col0 + 512 * j, K);
        if constexpr (kScaled) load_even(c[j], p.c, col0 + 512 * j, K);
      } else {
        load_piece(x[j], xrow, col0 + 512 * j, K, false);
        if constexpr (kGate) load_piece(g[j], grow, col0 + 512 * j, K, false);
        if constexpr (kScaled) load_piece(c[j], p.c, col0 + 512 * j, K, false);
      }
    }
  }
  __device__ __forceinline__ void values(const Mx4Rows& p, int col0, float (&v)[2][8]) const {
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
      if constexpr (kScaled) {
        float a[8];
        c[j].get(a);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] *= a[k];
      }
    }
    if (kEven && col0 + kRowBlock > (int)p.K) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[j][k] = col0 + 512 * j + (int)row_lane8() < (int)p.K ? v[j][k] : 0.0f;
    }
  }
};
// T: of the factor 1 / sqrt(hb) the power of two 2^-ceil(log2(hb) / 2) goes into the
// values, exactly, so that sums pass the largest float only where (nearly) a result does,
// and the sqrt(2) that an odd log2 hb leaves multiplies the results, one rounding of each.
// (1 / sqrt(128) itself in front rounded every one of 128 inputs.) The stages go from
// neighbours to the farthest values, whatever hb, so that v is what the header says to the bit.
__device__ __forceinline__ void mx4_transform(const Mx4Rows& p, float (&v)[2][8]) {
  if (p.lhb == 0) return;
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) v[j][k] *= p.norm;
  if (p.lhb == 10) {
    // (bit 9, the pieces', behind bit 8: in the registers that bit 8 used and gives back.
    // In front of bit 3, where it costs nothing, 2048 x 28672 took 43 us, so 45.)
    fwht_stages(v, 9);
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      swap_back<32>(v[0][k], v[1][k]);
      const float x = v[0][k], y = v[1][k];
      v[0][k] = x + y;
      v[1][k] = x - y;
    }
    fwht_restore(v, 8);
    return;
  }
  fwht_stages(v, p.lhb);
  fwht_restore(v, p.lhb);
  if (p.lhb & 1) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= 1.41421356237309504880f;
  }
}

}  // namespace lq
