// Norms of queries and keys for each head with the rotation by position
// (include/lq.h gives the formulas).
//
// A lane holds 16 values of a head, 8 rotated pairs: of two halves 8 values
// each, of neighbours 16 in a row, so that no pair lies in two lanes; the
// values behind the rotated ones follow, 16 to a lane. 1 to 64 lanes make a
// head, whose sum of squares is a few lane exchanges, and a wavefront a group of
// heads. Wavefronts do not meet: each takes a part of one token's groups,
// computes the token's angles for itself (one to a lane, in fp64 up to their
// sines and cosines) and passes them round through LDS of its own, while its
// first groups are on their way. fp64 there, because position times frequency
// needs more than fp32 holds from a few thousand positions on.
//
// Bound by the bytes for many tokens: 2048 of 64 + 8 heads of 128, bf16, from memory,
// normed and rotated 17.2 us (4.4 TB/s of its 75 MB), rotated alone 15.2, fp32 29.2 (5.2);
// 777 of 40 + 8 heads of 80, fp32, 10.2. One token 3.0 us, with norms 3.6: the launch,
// a trip to memory and the angles. A workgroup to a token, whose wavefronts share
// the angles and so meet once, took 21.4 us where these took 17.6 in their first form.
#include "lq_qk.h"

#include "lq_rows.h"

namespace lq {
namespace {

// A lane's piece of a head: n values (at most 8) from `off` on.
struct Place {
  int off, n;
};
__device__ __forceinline__ Place place(int off, int end) { return {off, max(0, min(8, end - off))}; }

// Loaded at its element's alignment, those that do not exist as zero: 8 at
// once, or 4, 2 and 1 of them. Pieces hold a multiple of kGrain (8, 4 or 1): what
// that rules out is left out (777 tokens of 40 + 8 heads of 80, 60 rotated, fp32
// 12.3 us with all of it, 11.1 with 4).
typedef uint32_t __attribute__((ext_vector_type(4), aligned(2))) u32x4_u;
typedef uint32_t __attribute__((ext_vector_type(2), aligned(2))) u32x2_u;
typedef uint32_t __attribute__((aligned(2))) u32_u;
template <bool kBF16, int kGrain>
__device__ __forceinline__ void load8(RowPiece<kBF16>& to, const void* head, const Place& at) {
  const char* const p = reinterpret_cast<const char*>(head) + at.off * (kBF16 ? 2 : 4);
  const bool four = kGrain < 8 && (at.n & 4), pair = kGrain < 4 && (at.n & 2), odd = kGrain < 4 && (at.n & 1);
  if constexpr (kBF16) {
    u32x4_u all = {0, 0, 0, 0};
    if (at.n >= 8) all = *reinterpret_cast<const u32x4_u*>(p);
    if (kGrain < 8 && at.n < 8) {
      u32x2_u quad = {0, 0};
      uint32_t two = 0, one = 0;
      if (four) quad = *reinterpret_cast<const u32x2_u*>(p);
      if (pair) two = *reinterpret_cast<const u32_u*>(p + 2 * (at.n & 4));
      if (odd) one = *reinterpret_cast<const uint16_t*>(p + 2 * (at.n & 6));
      const uint32_t first = pair ? two : one, second = pair ? one : 0u;
      all = four ? (u32x4_u){quad[0], quad[1], first, second} : (u32x4_u){first, second, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) to.w[i] = all[i];
  } else {
    u32x4_u low = {0, 0, 0, 0}, high = {0, 0, 0, 0};
    if (at.n >= 4) low = *reinterpret_cast<const u32x4_u*>(p);
    if (at.n >= 8) high = *reinterpret_cast<const u32x4_u*>(p + 16);
    if (kGrain < 4 && at.n < 8) {
      u32x2_u two = {0, 0};
      uint32_t one = 0;
      if (pair) two = *reinterpret_cast<const u32x2_u*>(p + 4 * (at.n & 4));
      if (odd) one = *reinterpret_cast<const uint32_t*>(p + 4 * (at.n & 6));
      const u32x4_u rest = {pair ? two[0] : one, two[1], pair ? one : 0u, 0};
      if (four) high = rest;
      else low = rest;
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) to.w[i] = low[i], to.w[4 + i] = high[i];
  }
}
template <bool kBF16, int kGrain>
__device__ __forceinline__ void store8(void* head, const Place& at, const float (&v)[8]) {
  char* p = reinterpret_cast<char*>(head) + at.off * (kBF16 ? 2 : 4);
  if constexpr (kBF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
    if (at.n >= 8) {
      __builtin_memcpy(p, w, 16);
    } else if constexpr (kGrain < 8) {
      if (at.n & 4) {
        __builtin_memcpy(p, w, 8);
        p += 8;
        w[0] = w[2];
        w[1] = w[3];
      }
      if (kGrain < 4 && (at.n & 2)) {
        __builtin_memcpy(p, w, 4);
        p += 4;
        w[0] = w[1];
      }
      if (kGrain < 4 && (at.n & 1)) *reinterpret_cast<uint16_t*>(p) = (uint16_t)w[0];
    }
  } else {
    typedef float __attribute__((ext_vector_type(4), aligned(4))) f32x4_u;
    if (at.n >= 8) {
      *reinterpret_cast<f32x4_u*>(p) = (f32x4_u){v[0], v[1], v[2], v[3]};
      *reinterpret_cast<f32x4_u*>(p + 16) = (f32x4_u){v[4], v[5], v[6], v[7]};
    } else if constexpr (kGrain == 4) {
      if (at.n & 4) *reinterpret_cast<f32x4_u*>(p) = (f32x4_u){v[0], v[1], v[2], v[3]};
    } else if constexpr (kGrain < 4) {
      typedef float __attribute__((ext_vector_type(2), aligned(4))) f32x2_u;
      const bool four = at.n & 4, pair = at.n & 2;
      // (values, which the compiler would otherwise choose by their address)
      float w[7];
#pragma unroll
      for (int i = 0; i < 7; ++i) {
        w[i] = v[i];
        asm("" : "+v"(w[i]));
      }
      if (four) *reinterpret_cast<f32x4_u*>(p) = (f32x4_u){w[0], w[1], w[2], w[3]};
      if (pair) *reinterpret_cast<f32x2_u*>(p + 4 * (at.n & 4)) = four ? (f32x2_u){w[4], w[5]} : (f32x2_u){w[0], w[1]};
      if (at.n & 1)
        *reinterpret_cast<float*>(p + 4 * (at.n & 6)) = four ? (pair ? w[6] : w[4]) : pair ? w[2] : w[0];
    }
  }
}

// The sum over the 2^lanes_log lanes of a head.
__device__ __forceinline__ float head_sum(float v, int lanes_log) {
  if (lanes_log > 0) v += lane_xor<1>(v);
  if (lanes_log > 1) v += lane_xor<2>(v);
  if (lanes_log > 2) v += lane_xor<4>(v);
  if (lanes_log > 3) v += lane_xor<8>(v);
  if (lanes_log > 4) v += lane_xor<16>(v);
  if (lanes_log > 5) v += lane_xor<32>(v);
  return v;
}

// cos and sin of an angle in fp64, each rounded once: the angle in turns less whole and
// quarter turns, which is exact, and of the rest, at most pi / 4, the Taylor sums up to
// r^11 and r^10 (what follows is below 2^-37 and 2^-33). The fraction of a turn as a
// float, and sine and cosine of that, were off by up to 1e-7, at the same cost but
// for 2% (2048 tokens of 64 + 8 heads of 128 16.9 us, 17.2 so; one token 3.0 either way).
__device__ __forceinline__ void turn_of(double angle, float& c, float& s) {
  double t = angle * 0.15915494309189533577;
  t -= rint(t);
  const double q = rint(4.0 * t), r = fma(-0.25, q, t) * 6.28318530717958647693, z = r * r;
  double a = fma(z, -1.0 / 39916800.0, 1.0 / 362880.0), b = fma(z, -1.0 / 3628800.0, 1.0 / 40320.0);
  a = fma(z, a, -1.0 / 5040.0);
  b = fma(z, b, -1.0 / 720.0);
  a = fma(z, a, 1.0 / 120.0);
  b = fma(z, b, 1.0 / 24.0);
  a = fma(z, a, -1.0 / 6.0);
  b = fma(z, b, -0.5);
  const float sr = (float)fma(r * z, a, r), cr = (float)fma(z, b, 1.0);
  const int quarter = (int)q;            // -2 .. 2
  const float cq = quarter & 1 ? sr : cr, sq = quarter & 1 ? cr : sr;
  c = (quarter + 1) & 2 ? -cq : cq;
  s = quarter & 2 ? -sq : sq;
}

constexpr int kBatch = 1;        // groups on their way together, and as many behind them

template <bool kBF16, bool kInterleaved, int kGrain>
__global__ __launch_bounds__(256) void qk_norm_rope_kernel(QkNormRope p, int lanes_log, int parts) {
  __shared__ float turns[4][2][kQkMaxDim / 2];
  const int64_t unit = (int64_t)blockIdx.x * 4 + wave_id();
  const int64_t b = unit / parts;
  if (b >= p.B) return;
  const int part = (int)(unit - b * parts);
  float (&turn)[2][kQkMaxDim / 2] = turns[wave_id()];
  constexpr int kSize = kBF16 ? 2 : 4;
  const int lane = threadIdx.x & 63, half = p.rot / 2;
  const int per = 64 >> lanes_log;                       // heads of a group
  const int j = lane & ((1 << lanes_log) - 1), h_in = lane >> lanes_log;
  const int rl = (p.rot + 15) / 16;                      // lanes that rotate
  const bool rotates = j < rl;
  Place at[2];
  if (rotates && !kInterleaved) {
    at[0] = place(8 * j, half);
    at[1] = place(half + 8 * j, p.rot);
  } else {
    const int off = rotates ? 16 * j : p.rot + 16 * (j - rl), end = rotates ? p.rot : p.dim;
    at[0] = place(off, end);
    at[1] = place(off + 8, end);
  }
  const int qu = (p.part[0].heads + per - 1) / per, groups = qu + (p.part[1].heads + per - 1) / per;
  const int g0 = groups * part / parts, g1 = groups * (part + 1) / parts;

  RowPiece<kBF16> in[2][kBatch][2];
  auto head = [&](int g) __attribute__((always_inline)) { return (g < qu ? g : g - qu) * per + h_in; };
  auto load = [&](RowPiece<kBF16> (&to)[kBatch][2], int g) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < kBatch; ++i) {
      // (past the last group: that one again; heads past the last: the first)
      const int gi = min(g + i, g1 - 1);
      const QkHeads& t = p.part[gi < qu ? 0 : 1];
      const int h = head(gi) < t.heads ? head(gi) : 0;
      const char* const x = reinterpret_cast<const char*>(t.x) + (b * t.ld + h * t.ld_head) * kSize;
#pragma unroll
      for (int k = 0; k < 2; ++k) load8<kBF16, kGrain>(to[i][k], x, at[k]);
    }
  };
  // (the norms' weights too before the angles: behind them they were a trip to memory more)
  RowPiece<false> wp[2];
  auto load_weights = [&](const QkHeads& t) __attribute__((always_inline)) {
    if (t.w == nullptr) return;
#pragma unroll
    for (int i = 0; i < 2; ++i) load8<false, kGrain>(wp[i], t.w, at[i]);
  };
  load(in[0], g0);
  if (p.norm) load_weights(p.part[g0 < qu ? 0 : 1]);

  if (half > 0) {
    const double pos = p.pos64 ? (double)reinterpret_cast<const int64_t*>(p.pos)[b]
                               : (double)reinterpret_cast<const int32_t*>(p.pos)[b];
    for (int i = lane; i < half; i += 64) {
      turn_of(pos * p.freq[i], turn[0][i], turn[1][i]);
    }
    // (the wavefront's own stores, before its reads)
    __builtin_amdgcn_fence(__ATOMIC_RELEASE, "wavefront");
    __builtin_amdgcn_s_waitcnt(3 << 14 | 7 << 4 | 15);
    __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "wavefront");
  }
  float c[8], s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    // (places past the last angle: an angle of this token, whose product is dropped)
    c[k] = rotates ? turn[0][min(8 * j + k, half - 1)] : 1.0f;
    s[k] = rotates ? turn[1][min(8 * j + k, half - 1)] : 0.0f;
  }
  float w[2][8];
  auto take_weights = [&](const QkHeads& t) __attribute__((always_inline)) {
    const float plus = p.one_plus ? 1.0f : 0.0f;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      wp[i].get(w[i]);
#pragma unroll
      for (int k = 0; k < 8; ++k) w[i][k] = t.w != nullptr ? plus + w[i][k] : 1.0f;
    }
  };
  if (p.norm) take_weights(p.part[g0 < qu ? 0 : 1]);

  auto one = [&](const RowPiece<kBF16> (&piece)[2], int g) __attribute__((always_inline)) {
    if (g >= g1) return;
    const QkHeads& t = p.part[g < qu ? 0 : 1];
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) piece[i].get(v[i]);
    if (p.norm) {
      if (g == qu && g != g0) {
        load_weights(t);
        take_weights(t);
      }
      float q[2] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) q[i] = fmaf(v[i][k], v[i][k], q[i]);
      const float sum = head_sum(q[0] + q[1], lanes_log);
      const float mean = sum / (float)p.dim + p.eps;
      float r = inv_root(mean);
      // (the sum, or it and a large eps, passes the largest float)
      if (__builtin_amdgcn_ballot_w64(!(sum <= 3.0e38f && mean <= 3.4e38f)) != 0) {
        // (as norm_block.hip: squares of v 2^-80, half of that factor into v)
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float u = v[i][k] * 0x1p-80f;
            z = fmaf(u, u, z);
          }
        z = head_sum(z, lanes_log);
        if (!(sum <= 3.0e38f && mean <= 3.4e38f)) {
          r = inv_root(z / (float)p.dim + p.eps * 0x1p-80f * 0x1p-80f) * 0x1p-40f;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] *= 0x1p-40f;
        }
      }
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = v[i][k] * r * w[i][k];
    }
    if (rotates) {
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        float& a = kInterleaved ? v[k >> 2][2 * (k & 3)] : v[0][k];
        float& d = kInterleaved ? v[k >> 2][2 * (k & 3) + 1] : v[1][k];
        const float a0 = a, d0 = d;
        a = fmaf(a0, c[k], -(d0 * s[k]));
        d = fmaf(d0, c[k], a0 * s[k]);
      }
    }
    const int h = head(g);
    if (h < t.heads) {
      char* const o = reinterpret_cast<char*>(t.out) + (b * t.ldo + h * t.ldo_head) * kSize;
#pragma unroll
      for (int i = 0; i < 2; ++i) store8<kBF16, kGrain>(o, at[i], v[i]);
    }
  };
  for (int g = g0; g < g1; g += 2 * kBatch) {
    if (g + kBatch < g1) load(in[1], g + kBatch);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) one(in[0][i], g + i);
    if (g + 2 * kBatch < g1) load(in[0], g + 2 * kBatch);
#pragma unroll
    for (int i = 0; i < kBatch; ++i) one(in[1][i], g + kBatch + i);
  }
}

template <bool kBF16, int kGrain>
void enqueue(const QkNormRope& p, int lanes_log, int parts, dim3 grid, hipStream_t stream) {
  const dim3 block(256);
  if (p.interleaved)
    hipLaunchKernelGGL((qk_norm_rope_kernel<kBF16, true, kGrain>), grid, block, 0, stream, p, lanes_log, parts);
  else
    hipLaunchKernelGGL((qk_norm_rope_kernel<kBF16, false, kGrain>), grid, block, 0, stream, p, lanes_log, parts);
}
template <bool kBF16>
void enqueue(const QkNormRope& p, int lanes_log, int parts, dim3 grid, hipStream_t stream) {
  // what every piece's values are a multiple of
  const int all = (p.interleaved ? p.rot : p.rot / 2) | (p.dim - p.rot);
  if (all % 8 == 0) enqueue<kBF16, 8>(p, lanes_log, parts, grid, stream);
  else if (all % 4 == 0) enqueue<kBF16, 4>(p, lanes_log, parts, grid, stream);
  else enqueue<kBF16, 1>(p, lanes_log, parts, grid, stream);
}

// Wavefronts that keep the device busy.
constexpr int64_t kWaves = 4096;

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRope& p, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const int lanes = (p.rot + 15) / 16 + (p.dim - p.rot + 15) / 16;
  int lanes_log = 0;
  while ((1 << lanes_log) < lanes) ++lanes_log;
  const int per = 64 >> lanes_log;
  const int groups = (p.part[0].heads + per - 1) / per + (p.part[1].heads + per - 1) / per;
  const int64_t want = kWaves / p.B;
  const int parts = want < 1 ? 1 : want < groups ? (int)want : groups;
  const dim3 grid((unsigned)((p.B * parts + 3) / 4));
  if (p.bf16) enqueue<true>(p, lanes_log, parts, grid, stream);
  else enqueue<false>(p, lanes_log, parts, grid, stream);
  return hipGetLastError();
}

}  // namespace lq
