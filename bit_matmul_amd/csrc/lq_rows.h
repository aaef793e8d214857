// Device helpers of the row kernels (quant_rows.hip, norm_block.hip): one
// workgroup holds one row of K values in registers. Device-only.
//
// Layout: the row is cut into blocks of 1024 values; wavefront w of W takes
// blocks w, w + W, ... (C of them). Of a block, lane l holds the values
// 8 l .. 8 l + 7 and 512 + 8 l .. 512 + 8 l + 7: a wavefront's loads are
// consecutive 16-byte pieces, its 8-bit stores consecutive 8-byte ones, and
// the index bits of a block are three register bits, six lane bits and one
// register bit, so a Hadamard block of up to 1024 needs no LDS.
#pragma once

#include "lq_internal.h"
#include "lq_prep.h"

namespace lq {

constexpr int kRowBlock = 1024;
constexpr int kRowMaxWaves = 16;
constexpr int kRowMaxC = 4;
constexpr int64_t kRowMaxK = (int64_t)kRowBlock * kRowMaxWaves * kRowMaxC;

// Values p[0..7] as floats, those past n (n may be <= 0) as zero. p needs
// only its element's alignment: gfx950's global loads take any byte address,
// and one 16-byte load is one instruction for an odd row stride too.
template <bool kBF16>
__device__ __forceinline__ void load_row8(const void* base, int64_t at, int n, float (&v)[8]) {
  if constexpr (kBF16) {
    const uint16_t* p = reinterpret_cast<const uint16_t*>(base) + at;
    if (n >= 8) {
      uint32_t w[4];
      __builtin_memcpy(w, p, 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? bf16_bits_to_f32(p[i]) : 0.0f;
    }
  } else {
    const float* p = reinterpret_cast<const float*>(base) + at;
    if (n >= 8) {
      __builtin_memcpy(v, p, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = i < n ? p[i] : 0.0f;
    }
  }
}

__device__ __forceinline__ void store_row8(void* base, bool bf16, int64_t at, int n,
                                           const float (&v)[8]) {
  if (bf16) {
    uint16_t* p = reinterpret_cast<uint16_t*>(base) + at;
    if (n >= 8) {
      uint32_t w[4];
#pragma unroll
      for (int i = 0; i < 4; ++i)
        w[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
      __builtin_memcpy(p, w, 16);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = (uint16_t)f32_to_bf16_bits(v[i]);
    }
  } else {
    float* p = reinterpret_cast<float*>(base) + at;
    if (n >= 8) {
      __builtin_memcpy(p, v, 32);
    } else {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) p[i] = v[i];
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
  __syncthreads();
  v = (lane & 15) < waves ? lds[lane & 15] : Op::id();
  v = Op::of(v, lane_xor<1>(v));
  v = Op::of(v, lane_xor<2>(v));
  v = Op::of(v, lane_xor<4>(v));
  return Op::of(v, lane_xor<8>(v));
}

// ------------------------------------------------------------ activations
// The values of lq_act (include/lq.h).
constexpr int kActNone = 0, kActSilu = 1, kActGelu = 2, kActSigmoid = 3, kActTanh = 4;

// 1 / (1 + exp(-x)) to a few units in the last place: exp as the hardware's
// power of two of x log2(e), whose product is carried in two floats (one
// float would lose |x| units), and one Newton step on the hardware's
// reciprocal. Below -80 the value of -80 (2e-35) stands for what would
// overflow the exponential.
__device__ __forceinline__ float sigmoid_f32(float x) {
  constexpr float kLog2e = 1.44269504088896340736f, kLog2eLo = 1.92596299112661746887e-8f;
  const float m = x < -80.0f ? 80.0f : -x;
  const float hi = m * kLog2e;
  const float lo = fmaf(m, kLog2e, -hi) + m * kLog2eLo;
  // m of -inf (x = +inf): lo is NaN and exp2 of hi is zero
  float e = __builtin_amdgcn_exp2f(hi);
  e = hi > -126.0f ? fmaf(e, lo * 0.69314718055994530942f, e) : e;
  const float d = 1.0f + e;
  const float r = __builtin_amdgcn_rcpf(d);
  return fmaf(r, fmaf(-d, r, 1.0f), r);
}

__device__ __forceinline__ float gelu_tanh_f32(float g) {
  // 0.5 g (1 + tanh(u)) = g / (1 + exp(-2 u)), u = sqrt(2 / pi) (g + 0.044715 g^3)
  return g * sigmoid_f32(1.59576912160573071176f * fmaf(0.044715f * g * g, g, g));
}

__device__ __forceinline__ void act_row8(int act, float (&g)[8]) {
  switch (act) {
    case kActSilu:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] *= sigmoid_f32(g[i]);
      break;
    case kActGelu:
#pragma unroll
      for (int i = 0; i < 8; ++i) g[i] = gelu_tanh_f32(g[i]);
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

// ------------------------------------------------------------ 8-bit codes
// The codes of a row: q = v 127 / top rounded to the nearest whole number,
// ties to even, decided as the real quotient decides it, not as a rounded
// one does.
struct RowCoder {
  float top, lift, r;
  bool bad;          // the row holds an infinity or a NaN: codes 0, scale NaN
  __device__ __forceinline__ explicit RowCoder(float max_bits) {
    bad = __float_as_uint(max_bits) >= 0x7F800000u;
    // 127 / top overflows below 2^-121: such rows are lifted by 2^100 first
    lift = max_bits < 0x1p-100f ? 0x1p100f : 1.0f;
    top = max_bits * lift;
    r = bad || max_bits == 0.0f ? 0.0f : 127.0f / top;
  }
  __device__ __forceinline__ float scale(float max_bits) const {
    return bad ? __uint_as_float(0x7FC00000u) : max_bits / 127.0f;
  }
  // v r is within 2 roundings of a value of at most 127, 1.6e-5, of the
  // quotient: only a product nearer than that to a half is decided by the
  // quotient itself, in 64 bits (127 v is exact there and a quotient of
  // floats that is no tie is further than 2^-33 from one).
  __device__ __forceinline__ uint2 codes(const float (&v)[8]) const {
    float q[8];
    bool near = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float t = v[i] * lift * r;
      q[i] = rintf(t);
      near = near || fabsf(t - q[i]) > 0.49997f;
    }
    if (near) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        q[i] = (float)rint((double)(v[i] * lift) * 127.0 / (double)top);
    }
    uint32_t w[2] = {0, 0};
    if (!bad) {
#pragma unroll
      for (int i = 0; i < 8; ++i) w[i >> 2] |= ((uint32_t)(int)q[i] & 0xFFu) << (8 * (i & 3));
    }
    return make_uint2(w[0], w[1]);
  }
};

// One 8-code piece of a row at column s (a multiple of 8) of K: written where
// it lies below K rounded up to 16, so the row's pad to 16 holds zeros.
__device__ __forceinline__ void store_codes(int8_t* q, int64_t row_at, int64_t s, int64_t K,
                                            uint2 w) {
  if (s < ((K + 15) & ~(int64_t)15)) *reinterpret_cast<uint2*>(q + row_at + s) = w;
}

}  // namespace lq
