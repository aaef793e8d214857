// 4-bit product y[b][n] = row_scale[n] sum_k q[b][k] w[n][k] + bias[n] of
// microscaled rows (include/lq.h gives the format),
// v_mfma_scale_f32_16x16x128_f8f6f4: lane (g, r) holds block 4 s + g of row r
// of a panel for product s, 16 bytes, and its scale byte. 16 weight rows x 16
// tokens to a wavefront, operands straight from memory.
#include "lq_mx4.h"

namespace lq {
namespace {

typedef __attribute__((ext_vector_type(4))) float f32x4;
typedef __attribute__((ext_vector_type(8))) int i32x8;

__global__ __launch_bounds__(256) void mx4_plain_kernel(Mx4Gemm p) {
  const int lane = threadIdx.x & 63, g = lane >> 4, r = lane & 15;
  const int64_t n0 = ((int64_t)blockIdx.x * 4 + wave_id()) * 16;
  if (n0 >= p.N) return;
  const int blocks = (int)((p.K + kMxBlock - 1) / kMxBlock), units = (int)mx4_units(p.K);
  const uint8_t* const wrow = p.w + min(n0 + r, p.N - 1) * p.ldw;
  const uint8_t* const wsc = p.w_scale + (n0 / 16) * units * 128 + 8 * r + 2 * g;
  for (int64_t b0 = (int64_t)blockIdx.y * 16; b0 < p.B; b0 += (int64_t)gridDim.y * 16) {
    const uint8_t* const qrow = p.q + min(b0 + r, p.B - 1) * p.ldq;
    const uint8_t* const qsc = p.scale + (b0 / 16) * units * 128 + 8 * r + 2 * g;
    f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
    for (int s = 0; 4 * s < blocks; ++s) {
      const int blk = 4 * s + g;
      i32x8 a = {}, c = {};
      int sa = 127, sc = 127;
      if (blk < blocks) {
        const uint4 wa = *reinterpret_cast<const uint4*>(wrow + 16 * blk);
        const uint4 qa = *reinterpret_cast<const uint4*>(qrow + 16 * blk);
        sa = wsc[(s >> 1) * 128 + (s & 1)];
        sc = qsc[(s >> 1) * 128 + (s & 1)];
        a[0] = (int)wa.x; a[1] = (int)wa.y; a[2] = (int)wa.z; a[3] = (int)wa.w;
        c[0] = (int)qa.x; c[1] = (int)qa.y; c[2] = (int)qa.z; c[3] = (int)qa.w;
        const int left = (int)p.K - 32 * blk;      // of these 32 codes, those that count
#pragma unroll
        for (int i = 0; i < 4; ++i)
          c[i] &= left >= 8 * i + 8 ? -1 : left <= 8 * i ? 0 : (int)((1u << (4 * (left - 8 * i))) - 1u);
      }
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(a, c, acc, 4, 4, 0, sa, 0, sc);
    }
    const int64_t b = b0 + r;
    if (b >= p.B) continue;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int64_t n = n0 + 4 * g + e;
      if (n >= p.N) continue;
      const float v = fmaf(acc[e], p.row_scale ? p.row_scale[n] : 1.0f, p.bias ? p.bias[n] : 0.0f);
      if (p.y_bf16) reinterpret_cast<uint16_t*>(p.y)[b * p.ldy + n] = (uint16_t)f32_to_bf16_bits(v);
      else reinterpret_cast<float*>(p.y)[b * p.ldy + n] = v;
    }
  }
}

}  // namespace

Mx4Plan plan_mx4(int64_t B, int64_t N, int64_t K, int cus) {
  return {64, 16, 1, (int)((N + 63) / 64), 0};
}

hipError_t launch_mx4_gemm(const Mx4Gemm& p, const Mx4Plan& plan, float* partial, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const int64_t tb = (p.B + 15) / 16;
  hipLaunchKernelGGL(mx4_plain_kernel, dim3((unsigned)plan.tiles, (unsigned)(tb < 1024 ? tb : 1024)), dim3(256), 0,
                     stream, p);
  return hipGetLastError();
}

}  // namespace lq
