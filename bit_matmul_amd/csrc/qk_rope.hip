// Norms of queries and keys for each head with the rotation by position
// (include/lq.h gives the formulas), one token to a workgroup.
//
// A lane holds 16 values of a head, 8 rotated pairs: of two halves 8 values
// each, of neighbours 16 in a row, so that no pair lies in two lanes; the
// values behind the rotated ones follow, 16 to a lane. 1 to 64 lanes make a
// head, whose sum of squares is a few lane exchanges. The token's angles are
// computed once by the workgroup, in fp64 up to their fraction of a turn, and
// read from LDS.
#include "lq_qk.h"

#include "lq_rows.h"

namespace lq {
namespace {

// 8 values at p (at its element's alignment), those from n on as zero.
template <bool kBF16, bool kWhole>
__device__ __forceinline__ void load8(const void* p, int n, float (&v)[8]) {
  RowPiece<kBF16> w;
#pragma unroll
  for (int i = 0; i < (kBF16 ? 4 : 8); ++i) w.w[i] = 0;
  if (n >= 8) {
    __builtin_memcpy(w.w, p, sizeof(w.w));
  } else if constexpr (!kWhole) {
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (kBF16) w.w[i / 2] |= (uint32_t)reinterpret_cast<const uint16_t*>(p)[i] << (16 * (i & 1));
        else w.w[i] = reinterpret_cast<const uint32_t*>(p)[i];
      }
  }
  w.get(v);
}
template <bool kBF16, bool kWhole>
__device__ __forceinline__ void store8(void* p, int n, const float (&v)[8]) {
  if constexpr (kBF16) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) w[i] = f32_to_bf16_bits(v[2 * i]) | (f32_to_bf16_bits(v[2 * i + 1]) << 16);
    if (n >= 8) {
      __builtin_memcpy(p, w, 16);
    } else if constexpr (!kWhole) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) reinterpret_cast<uint16_t*>(p)[i] = (uint16_t)(w[i / 2] >> (16 * (i & 1)));
    }
  } else {
    if (n >= 8) {
      __builtin_memcpy(p, v, 32);
    } else if constexpr (!kWhole) {
#pragma unroll
      for (int i = 0; i < 8; ++i)
        if (i < n) reinterpret_cast<float*>(p)[i] = v[i];
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

template <bool kBF16, bool kInterleaved, bool kWhole>
__global__ __launch_bounds__(1024) void qk_norm_rope_kernel(QkNormRope p, int lanes_log) {
  __shared__ float turn[2][kQkMaxDim / 2];
  const int64_t b = blockIdx.x;
  const int half = p.rot / 2;
  for (int i = threadIdx.x; i < kQkMaxDim / 2; i += (int)blockDim.x) {
    float s = 0.0f, c = 1.0f;
    if (i < half) {
      const double at = p.pos64 ? (double)reinterpret_cast<const int64_t*>(p.pos)[b]
                                : (double)reinterpret_cast<const int32_t*>(p.pos)[b];
      double t = at * p.freq[i] * 0.15915494309189533577;      // turns
      t -= rint(t);
      sincospif(2.0f * (float)t, &s, &c);
    }
    turn[0][i] = c;
    turn[1][i] = s;
  }
  __syncthreads();
  constexpr int kSize = kBF16 ? 2 : 4;
  const int lane = threadIdx.x & 63;
  const int per = 64 >> lanes_log;                       // heads of a wavefront
  const int j = lane & ((1 << lanes_log) - 1), h_in = lane >> lanes_log;
  const int rl = (p.rot + 15) / 16;                      // lanes that rotate
  const bool rotates = j < rl;
  int off[2], n[2];
  if (rotates && !kInterleaved) {
    off[0] = 8 * j;
    off[1] = half + 8 * j;
    n[0] = n[1] = min(8, half - 8 * j);
  } else {
    const int end = rotates ? p.rot : p.dim;
    off[0] = rotates ? 16 * j : p.rot + 16 * (j - rl);
    off[1] = off[0] + 8;
    n[0] = max(0, min(8, end - off[0]));
    n[1] = max(0, min(8, end - off[1]));
  }
  float c[8], s[8];
#pragma unroll
  for (int k = 0; k < 8; ++k) {
    c[k] = rotates ? turn[0][min(8 * j + k, kQkMaxDim / 2 - 1)] : 1.0f;
    s[k] = rotates ? turn[1][min(8 * j + k, kQkMaxDim / 2 - 1)] : 0.0f;
  }
  const int qu = (p.part[0].heads + per - 1) / per, units = qu + (p.part[1].heads + per - 1) / per;
  for (int u = wave_id(); u < units; u += (int)blockDim.x >> 6) {
    const QkHeads& t = p.part[u < qu ? 0 : 1];
    const int h = (u < qu ? u : u - qu) * per + h_in;
    const bool mine = h < t.heads;
    const char* const x = reinterpret_cast<const char*>(t.x) + (b * t.ld + (mine ? h : 0) * t.ld_head) * kSize;
    char* const o = reinterpret_cast<char*>(t.out) + (b * t.ldo + (mine ? h : 0) * t.ldo_head) * kSize;
    float v[2][8];
#pragma unroll
    for (int i = 0; i < 2; ++i) load8<kBF16, kWhole>(x + off[i] * kSize, n[i], v[i]);
    if (p.norm) {
      float q[2] = {};
#pragma unroll
      for (int i = 0; i < 2; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) q[i] = fmaf(v[i][k], v[i][k], q[i]);
      const float sum = head_sum(q[0] + q[1], lanes_log);
      float r = inv_root(sum / (float)p.dim + p.eps);
      if (__builtin_amdgcn_ballot_w64(!(sum <= 3.0e38f)) != 0) {
        // (as norm_block.hip: squares of v 2^-80, half of that factor into v)
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const float w = v[i][k] * 0x1p-80f;
            z = fmaf(w, w, z);
          }
        z = head_sum(z, lanes_log);
        if (!(sum <= 3.0e38f)) {
          r = inv_root(z / (float)p.dim + p.eps * 0x1p-80f * 0x1p-80f) * 0x1p-40f;
#pragma unroll
          for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int k = 0; k < 8; ++k) v[i][k] *= 0x1p-40f;
        }
      }
      const float plus = p.one_plus ? 1.0f : 0.0f;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        float w[8];
        if (t.w != nullptr) load8<false, kWhole>(t.w + off[i], n[i], w);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][k] = v[i][k] * r * (t.w != nullptr ? plus + w[k] : 1.0f);
      }
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
    if (mine) {
#pragma unroll
      for (int i = 0; i < 2; ++i) store8<kBF16, kWhole>(o + off[i] * kSize, n[i], v[i]);
    }
  }
}

template <bool kBF16>
void enqueue(const QkNormRope& p, bool whole, int lanes_log, dim3 grid, dim3 block, hipStream_t stream) {
  if (p.interleaved) {
    if (whole) hipLaunchKernelGGL((qk_norm_rope_kernel<kBF16, true, true>), grid, block, 0, stream, p, lanes_log);
    else hipLaunchKernelGGL((qk_norm_rope_kernel<kBF16, true, false>), grid, block, 0, stream, p, lanes_log);
  } else {
    if (whole) hipLaunchKernelGGL((qk_norm_rope_kernel<kBF16, false, true>), grid, block, 0, stream, p, lanes_log);
    else hipLaunchKernelGGL((qk_norm_rope_kernel<kBF16, false, false>), grid, block, 0, stream, p, lanes_log);
  }
}

}  // namespace

hipError_t launch_qk_norm_rope(const QkNormRope& p, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const int lanes = (p.rot + 15) / 16 + (p.dim - p.rot + 15) / 16;
  int lanes_log = 0;
  while ((1 << lanes_log) < lanes) ++lanes_log;
  const int per = 64 >> lanes_log;
  const int units = (p.part[0].heads + per - 1) / per + (p.part[1].heads + per - 1) / per;
  const bool whole = p.rot % 16 == 0 && p.dim % 16 == 0;
  const dim3 grid((unsigned)p.B), block(64u * (unsigned)(units < 16 ? units : 16));
  if (p.bf16) enqueue<true>(p, whole, lanes_log, grid, block, stream);
  else enqueue<false>(p, whole, lanes_log, grid, block, stream);
  return hipGetLastError();
}

}  // namespace lq
