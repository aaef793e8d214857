// Device helpers of the row kernels (quant_rows.hip, norm_block.hip): one
// workgroup holds one row of K values in registers. Parts of them serve
// mx4_rows.hip, mx4_token.hip, qk_rope.hip and int8_token.hip. Device-only.
//
// Layout: the row is cut into blocks of 1024 values; wavefront w of W takes
// blocks w, w + W, ... (C of them). Of a block, lane l holds the values
// 8 l .. 8 l + 7 and 512 + 8 l .. 512 + 8 l + 7: a wavefront's loads are
// consecutive 16-byte pieces in the order of its lanes, its 8-bit stores
// consecutive 8-byte ones, and the index bits of a block are three register
// bits, six lane bits and one register bit, so a Hadamard block of up to 1024
// needs no LDS.
#pragma once

#include "lq_8bit.h"
#include "lq_prep.h"

namespace lq {

// Piece j (0, 1) of a thread's block i begins at column row_col(i, j), the
// same for the wavefront, plus row_lane8(); row_whole: a wavefront's C blocks
// lie inside the row, so that none of its pieces is cut.
__device__ __forceinline__ int row_col(int i, int j) {
  return (wave_id() + i * ((int)blockDim.x >> 6)) * kRowBlock + 512 * j;
}
__device__ __forceinline__ uint32_t row_lane8() { return 8u * (threadIdx.x & 63u); }
template <int C>
__device__ __forceinline__ bool row_whole(int K) {
  return (wave_id() + (C - 1) * ((int)blockDim.x >> 6) + 1) * kRowBlock <= K;
}

// A piece of 8 values as it lies in memory. Loads fill these and nothing
// more, so that a wavefront has all of its loads in flight: converted where
// they are loaded (behind a test for the row's end or for a tensor that may
// be missing), each would wait for its own.
template <bool kBF16>
struct RowPiece {
  uint32_t w[kBF16 ? 4 : 8];
  __device__ __forceinline__ void get(float (&v)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      v[i] = __uint_as_float(!kBF16 ? w[i] : i % 2 ? w[i / 2] & 0xFFFF0000u : w[i / 2] << 16);
  }
};
// The piece at column col (of the wavefront) of a row of K values, those past
// K as zero. The row needs only its element's alignment: gfx950's global
// loads take any byte address, and 16 bytes are one load for an odd row
// stride too. (A scalar address plus a lane's offset: vector addresses of
// every piece of every tensor would take most of a long row's registers.)
template <bool kBF16>
__device__ __forceinline__ void load_piece(RowPiece<kBF16>& p, const void* row, int col, int K, bool whole) {
  constexpr uint32_t kSize = kBF16 ? 2 : 4;
  const char* from = reinterpret_cast<const char*>(row) + (int64_t)col * kSize;
  const uint32_t lane = row_lane8() * kSize;
  if (whole) {
    __builtin_memcpy(p.w, from + lane, sizeof(p.w));
    return;
  }
  const int n = K - col - (int)row_lane8();
#pragma unroll
  for (int i = 0; i < (kBF16 ? 4 : 8); ++i) p.w[i] = 0;
  if (n >= 8) {
    __builtin_memcpy(p.w, from + lane, sizeof(p.w));
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (kBF16) p.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(from + lane)[i] << (16 * (i & 1));
        else p.w[i] = reinterpret_cast<const uint32_t*>(from + lane)[i];
      }
  }
}

__device__ __forceinline__ void store_row8(void* row, bool bf16, int col, int K, bool whole,
                                           const float (&v)[8]) {
  char* const to = reinterpret_cast<char*>(row) + (int64_t)col * (bf16 ? 2 : 4);
  const int n = K - col - (int)row_lane8();
  if (bf16) {
    char* const p = to + row_lane8() * 2u;
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      w[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
    if (whole || n >= 8) {
      __builtin_memcpy(p, w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
    char* const p = to + row_lane8() * 4u;
    if (whole || n >= 8) {
      __builtin_memcpy(p, v, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) reinterpret_cast<float*>(p)[i] = v[i];
    }
  }
}

// ------------------------------------------------------------ reductions
struct SumF {
  static __device__ __forceinline__ float id() { return 0.0f; }
  static __device__ __forceinline__ float of(float a, float b) { return a + b; }
};
// Largest magnitude as a bit pattern: infinities and NaNs are above every
// finite value, so a row that holds one is seen in its maximum.
struct MaxBits {
  static __device__ __forceinline__ float id() { return 0.0f; }
  static __device__ __forceinline__ float of(float a, float b) {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    return __uint_as_float(x > y ? x : y);
  }
};

// Op over the workgroup, the same value in every thread. `lds` holds
// kRowMaxWaves floats that no other reduction of the kernel uses. The order
// is fixed: lanes by a butterfly, then the wavefronts' values by another.
template <typename Op>
__device__ __forceinline__ float row_reduce(float v, float* lds) {
  v = Op::of(v, lane_xor<1>(v));
  v = Op::of(v, lane_xor<2>(v));
  v = Op::of(v, lane_xor<4>(v));
  v = Op::of(v, lane_xor<8>(v));
  v = Op::of(v, lane_xor<16>(v));
  v = Op::of(v, lane_xor<32>(v));
  const int waves = (int)blockDim.x >> 6;
  if (waves == 1) return v;
  const int lane = threadIdx.x & 63;
  if (lane == 0) lds[threadIdx.x >> 6] = v;
  // (A barrier for LDS alone: __syncthreads would wait for the loads in flight.)
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
  __builtin_amdgcn_s_waitcnt(3 << 14 | 7 << 4 | 15);
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  v = (lane & 15) < waves ? lds[lane & 15] : Op::id();
  v = Op::of(v, lane_xor<1>(v));
  v = Op::of(v, lane_xor<2>(v));
  v = Op::of(v, lane_xor<4>(v));
  return Op::of(v, lane_xor<8>(v));
}

// 1 / sqrt(t), rounded once: the quotient of the root is off by a rounding of
// either, and its residual 1 - t r^2, exact but for its own last rounding,
// takes that out. (An infinite t has no residual: 0.)
__device__ __forceinline__ float inv_root(float t) {
  const float r = 1.0f / sqrtf(t);
  const float h = t * r, lo = fmaf(t, r, -h);
  const float e = fmaf(-lo, r, fmaf(-h, r, 1.0f));
  return __float_as_uint(t) < 0x7F800000u ? fmaf(0.5f * r, e, r) : r;
}

// ------------------------------------------------------------ activations
// The values of lq_act (include/lq.h).
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActSigmoid = 3, kActTanh = 4;

// 1 / (1 + exp(-x)) to a few units in the last place, from e = exp(-|x|),
// which cannot overflow: 1 / (1 + e), and e times it where x is negative (so
// that a large x times it vanishes as it should). exp is the hardware's power
// of two of x log2(e), whose product is carried in two floats (one float
// would lose |x| units); one Newton step on the hardware's reciprocal.
__device__ __forceinline__ float sigmoid_f32(float x) {
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLo = 1.92596299112661746887e-8f;
  const float m = -fabsf(x);
  const float hi = m * kLog2e;
  const float lo = fmaf(m, kLog2e, -hi) + m * kLog2eLo;
  // (hi of an infinite x: lo is NaN, exp2 of hi is zero. Where hi is below -126,
  // 1 + e is 1 and e itself counts for negative x only: shut_gate.)
  float e = __builtin_amdgcn_exp2f(hi);
  e = hi > -126.0f ? fmaf(e, lo * 0.69314718055994530942f, e) : e;
  const float d = 1.0f + e;
  float r = __builtin_amdgcn_rcpf(d);
  r = fmaf(r, fmaf(-d, r, 1.0f), r);
  return x < 0.0f ? e * r : r;
}

// Below kShut exp(x) comes near the floats below the normal ones, of which the
// hardware's power of two makes zeros, while x exp(x) is a normal float down to
// -91.9. m sigmoid(x) there is m exp(x), the power taken 2^64 times as large.
constexpr float kShut = -87.3f;
__device__ __forceinline__ float shut_gate(float x, float m) {
#pragma clang fp contract(off)      // (hi + 64 is a sum of hi as it was rounded: lo is what that lost)
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLo = 1.92596299112661746887e-8f;
  const float hi = x * kLog2e;
  const float lo = fmaf(x, kLog2e, -hi) + x * kLog2eLo;
  float e = __builtin_amdgcn_exp2f(hi + 64.0f);
  e = hi > -256.0f ? fmaf(e, lo * 0.69314718055994530942f, e) : e;
  return m * e * 0x1p-64f;
}

// The argument of gelu's sigmoid: 0.5 g (1 + tanh(u)) = g / (1 + exp(-2 u)),
// u = sqrt(2 / pi) (g + 0.044715 g^3). Above -9.9 it is above -85.1.
__device__ __forceinline__ float gelu_arg(float g) {
  return 1.59576912160573071176f * fmaf(0.044715f * g * g, g, g);
}

// act(g) of 8 values. Gates that shut as far as kShut are rare: one test of the
// 8 (bit patterns grow with a negative value's magnitude and are smaller for
// all others; a negative NaN takes the long way for nothing), and one branch
// for the three that have a sigmoid (2048 gated rows of 28672 66 -> 67 us; one
// in each of them was no faster).
__device__ __forceinline__ void act_row8(int act, float (&g)[8]) {
  const uint32_t shut = act == kActGelu ? __float_as_uint(-9.9f)
                        : act == kActSilu || act == kActSigmoid ? __float_as_uint(kShut) : ~0u;
  uint32_t most = __float_as_uint(g[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) most = max(most, __float_as_uint(g[i]));
  if (__builtin_amdgcn_ballot_w64(most > shut) != 0) {
    asm volatile("");      // (a branch)
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float x = act == kActGelu ? gelu_arg(g[i]) : g[i], m = act == kActSigmoid ? 1.0f : g[i];
      g[i] = x < kShut ? shut_gate(x, m) : m * sigmoid_f32(x);
      __builtin_amdgcn_sched_barrier(0);      // (one value's registers at a time)
    }
    return;
  }
  switch (act) {
    case kActSilu:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= sigmoid_f32(g[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= sigmoid_f32(gelu_arg(g[i]));
      break;
    case kActSigmoid:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = sigmoid_f32(g[i]);
      break;
    case kActTanh:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = tanhf(g[i]);
      break;
    default:
      break;
  }
}

// ------------------------------------------------------------ T
// A butterfly with lane ^ X (1, 2, 4, 8): a + p in the lane whose bit is clear,
// p - a in the other, as one fma with a multiplier of +-1. (With bound_ctrl
// the exchange needs no register cleared before it.)
template <int kDpp>
__device__ __forceinline__ float dpp(float v) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), kDpp, 0xF, 0xF, true));
}
template <int X>
__device__ __forceinline__ void dpp_stage(float (&a)[16], int lane) {
  const float sgn = (lane & X) != 0 ? -1.0f : 1.0f;
  float p[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) {
    if constexpr (X == 1) p[k] = dpp<0xB1>(a[k]);                // quad permutations
    else if constexpr (X == 2) p[k] = dpp<0x4E>(a[k]);
    else if constexpr (X == 4) p[k] = dpp<0x1B>(dpp<0x141>(a[k]));   // lane ^ 7, then ^ 3
    else p[k] = dpp<0x128>(a[k]);                                // 16 lanes rotated by 8
  }
#pragma unroll
  for (int k = 0; k < 16; ++k) a[k] = fmaf(a[k], sgn, p[k]);
}

// A butterfly over a lane bit (16 or 32) by exchanging it with register bit
// kReg: afterwards that register bit is the index bit and the lane bit holds
// what the register bit held. swap_back undoes it on the codes.
template <int kLaneBit>
__device__ __forceinline__ void lane_swap(uint32_t& x, uint32_t& y) {
  if constexpr (kLaneBit == 16) {
    const auto z = __builtin_amdgcn_permlane16_swap(x, y, false, false);
    x = z[0];
    y = z[1];
  } else {
    const auto z = __builtin_amdgcn_permlane32_swap(x, y, false, false);
    x = z[0];
    y = z[1];
  }
}
template <int kLaneBit, int kReg>
__device__ __forceinline__ void swap_stage(float (&a)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if ((k & kReg) == 0) {
      uint32_t x = __float_as_uint(a[k]), y = __float_as_uint(a[k | kReg]);
      lane_swap<kLaneBit>(x, y);
      a[k] = __uint_as_float(x) + __uint_as_float(y);
      a[k | kReg] = __uint_as_float(x) - __uint_as_float(y);
    }
}
template <int kReg>
__device__ __forceinline__ void reg_stage(float (&a)[16]) {
#pragma unroll
  for (int k = 0; k < 16; ++k)
    if ((k & kReg) == 0) {
      const float x = a[k], y = a[k | kReg];
      a[k] = x + y;
      a[k | kReg] = x - y;
    }
}

// The unnormalised Walsh-Hadamard transform of every 2^lhb values of a block.
// Index bits 0..2 and 9 are register bits, bits 3..8 lane bits; bits 7 and 8
// end up as register bits 2 and 3 (fwht_order puts the codes back).
__device__ __forceinline__ void fwht_stages(float (&v)[2][8], int lhb) {
  const int lane = threadIdx.x & 63;
  float a[16];
#pragma unroll
  for (int k = 0; k < 16; ++k) a[k] = v[k >> 3][k & 7];
  reg_stage<1>(a);
  if (lhb > 1) reg_stage<2>(a);
  if (lhb > 2) reg_stage<4>(a);
  if (lhb > 9) reg_stage<8>(a);
  if (lhb > 3) dpp_stage<1>(a, lane);
  if (lhb > 4) dpp_stage<2>(a, lane);
  if (lhb > 5) dpp_stage<4>(a, lane);
  if (lhb > 6) dpp_stage<8>(a, lane);
  if (lhb > 7) swap_stage<16, 4>(a);
  if (lhb > 8) swap_stage<32, 8>(a);
#pragma unroll
  for (int k = 0; k < 16; ++k) v[k >> 3][k & 7] = a[k];
}
// (The usual 1024 without a test between the stages, each of which would copy
// the 16 registers where its paths join.)
__device__ __forceinline__ void fwht_block(float (&v)[2][8], int lhb) {
  if (lhb == 10) fwht_stages(v, 10);
  else fwht_stages(v, lhb);
}
// w[j]: the codes of piece j (dword h: register bit 2 set).
__device__ __forceinline__ void fwht_order(uint2 (&w)[2], int lhb) {
  if (lhb > 8) {
    lane_swap<32>(w[0].x, w[1].x);
    lane_swap<32>(w[0].y, w[1].y);
  }
  if (lhb > 7) {
    lane_swap<16>(w[0].x, w[0].y);
    lane_swap<16>(w[1].x, w[1].y);
  }
}

// ------------------------------------------------------------ 8-bit codes
// The codes of a row: q = v 127 / top rounded to the nearest whole number,
// ties to even, decided as the real quotient decides it, not as a rounded
// one does.
struct RowCoder {
  float top, r;
  bool bad;          // the row holds an infinity or a NaN: codes 0, scale NaN
  bool tiny;         // 127 / top might overflow: every code by the quotient
  __device__ __forceinline__ explicit RowCoder(float max_bits) {
    top = max_bits;
    bad = __float_as_uint(max_bits) >= 0x7F800000u;
    tiny = max_bits > 0.0f && max_bits < 0x1p-100f;
    r = bad || tiny || max_bits == 0.0f ? 0.0f : 127.0f / max_bits;
  }
  __device__ __forceinline__ float scale(float norm) const {
    return bad ? __uint_as_float(0x7FC00000u) : top * norm / 127.0f;
  }
  // The codes of 8 values as two dwords. v r + 1.5 2^23 rounds v r to a whole
  // number, whose low byte is the sum's low byte. r is off by a rounding, so
  // that the product (at most 127) is off by at most 8e-6 from the quotient:
  // only one nearer than 1e-5 to a half is decided by the quotient itself, in
  // 64 bits (127 v is exact there, and a quotient of floats that is no tie is
  // further than 2^-33 from one).
  __device__ __forceinline__ uint2 codes(const float (&v)[8]) const {
    constexpr float kWhole = 12582912.0f;
    uint32_t u[8];
    float far = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float w = fmaf(v[i], r, kWhole);
      u[i] = __float_as_uint(w);
      far = fmaxf(far, fabsf(fmaf(v[i], r, kWhole - w)));
    }
    if (__builtin_amdgcn_ballot_w64(tiny || far > 0.49999f) != 0) {
      asm volatile("");      // (a branch: computed anyway and selected, it took half of the kernel's time)
#pragma unroll
      for (int i = 0; i < 8; ++i)
        u[i] = (uint32_t)(int)rint((double)v[i] * 127.0 / (double)top);
    }
    uint32_t o[2];
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const uint32_t lo = __builtin_amdgcn_perm(u[4 * h + 1], u[4 * h], 0x00000400u);
      const uint32_t hi = __builtin_amdgcn_perm(u[4 * h + 3], u[4 * h + 2], 0x00000400u);
      o[h] = bad ? 0u : __builtin_amdgcn_perm(hi, lo, 0x05040100u);
    }
    return make_uint2(o[0], o[1]);
  }
};

// The codes of the piece at column col of a row: written where they lie below
// K rounded up to 16, so the row's pad to 16 holds zeros.
__device__ __forceinline__ void store_codes(int8_t* row, int col, int K, uint2 w) {
  if (col + (int)row_lane8() < ((K + 15) & ~15)) *reinterpret_cast<uint2*>(row + col + row_lane8()) = w;
}

}  // namespace lq
