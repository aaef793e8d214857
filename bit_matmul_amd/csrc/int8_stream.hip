// 8-bit product y[b][n] = scale[b] row_scale[n] sum_k q[b][k] w[n][k] + bias[n]
// on v_mfma_i32_16x16x64_i8, exact 32-bit sums.
//
// A wavefront multiplies P panels of 16 weight rows with T tiles of 16 tokens
// over its share of the reduction; the wavefronts of a workgroup add their
// sums in LDS (whole numbers: any order gives the same sum).
//
// Operands straight from memory: lane 16 g + r brings the 16 bytes
// k = 64 s + 16 g .. + 15 of weight row r as A and of token r as B. Rows past
// N and tokens past B are read as the last one and never stored. K is taken
// up to the next multiple of 16 (the codes' pad is zero); the last 64-byte
// step past that is read as zero codes.
#include "lq_int8.h"

namespace lq {
namespace {

template <int P, int T>
__global__ __launch_bounds__(512) void int8_stream_kernel(Int8Gemm p, int tiles_n) {
  __shared__ int sum[P * T * 256];
  const int lane = threadIdx.x & 63, wave = wave_id(), waves = (int)blockDim.x >> 6;
  const int g = lane >> 4, r = lane & 15;
  const int64_t n0 = (int64_t)(blockIdx.x % tiles_n) * (16 * P);
  const int64_t b0 = (int64_t)(blockIdx.x / tiles_n) * (16 * T);
  for (int i = threadIdx.x; i < P * T * 256; i += blockDim.x) sum[i] = 0;

  const int8_t* wp[P];
  const int8_t* qp[T];
#pragma unroll
  for (int i = 0; i < P; ++i) wp[i] = p.w + min(n0 + 16 * i + r, p.N - 1) * p.ldw + 16 * g;
#pragma unroll
  for (int j = 0; j < T; ++j) qp[j] = p.q + min(b0 + 16 * j + r, p.B - 1) * p.ldq + 16 * g;
  const int K16 = ((int)p.K + 15) & ~15;
  const int steps = (K16 + 63) / 64, full = K16 / 64;
  const int lo = (int)((int64_t)steps * wave / waves), hi = (int)((int64_t)steps * (wave + 1) / waves);

  i32x4 acc[P][T];
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};
  const int end = min(hi, full);
  for (int s = lo; s < end; ++s) {
    i32x4 a[P], c[T];
#pragma unroll
    for (int i = 0; i < P; ++i) a[i] = *reinterpret_cast<const i32x4*>(wp[i] + 64 * (int64_t)s);
#pragma unroll
    for (int j = 0; j < T; ++j) c[j] = *reinterpret_cast<const i32x4*>(qp[j] + 64 * (int64_t)s);
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], c[j], acc[i][j], 0, 0, 0);
  }
  if (hi > full && hi == steps) {   // the last step ends inside its 64 bytes
    const bool in = 64 * full + 16 * g < K16;
    const int64_t at = in ? 64 * (int64_t)full : -16 * g;   // else the row's first bytes, codes zero
    i32x4 a[P], c[T];
#pragma unroll
    for (int i = 0; i < P; ++i) a[i] = *reinterpret_cast<const i32x4*>(wp[i] + at);
#pragma unroll
    for (int j = 0; j < T; ++j) {
      c[j] = *reinterpret_cast<const i32x4*>(qp[j] + at);
      if (!in) c[j] = (i32x4){0, 0, 0, 0};
    }
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int j = 0; j < T; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], c[j], acc[i][j], 0, 0, 0);
  }
  __syncthreads();
#pragma unroll
  for (int i = 0; i < P; ++i)
#pragma unroll
    for (int j = 0; j < T; ++j)
#pragma unroll
      for (int e = 0; e < 4; ++e) atomicAdd(&sum[((i * T + j) * 4 + e) * 64 + lane], acc[i][j][e]);
  __syncthreads();
  // lane (g, r) of tile (i, j): weight rows 4 g .. 4 g + 3 of the panel for token r
  for (int t = threadIdx.x; t < P * T * 64; t += blockDim.x) {
    const int i = (t >> 6) / T, j = (t >> 6) % T;
    const int64_t n = n0 + 16 * i + 4 * ((t >> 4) & 3), b = b0 + 16 * j + (t & 15);
    if (b >= p.B) continue;
    if (n >= p.N) continue;
    i32x4 v;
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = sum[((t >> 6) * 4 + e) * 64 + (t & 63)];
    float rs[4], bias[4];
    load_int8_rows(p, n, rs, bias);
    store_int8_sums(p, b, n, p.scale[b], rs, bias, v);
  }
}

}  // namespace

hipError_t launch_int8_gemm(const Int8Gemm& p, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const int64_t tiles_n = (p.N + 15) / 16;
  if (p.B > 64) return launch_int8_tile(p, stream);
  if (p.B <= 16) {
    hipLaunchKernelGGL((int8_stream_kernel<1, 1>), dim3((unsigned)tiles_n), dim3(512), 0, stream, p,
                       (int)tiles_n);
  } else {
    const int64_t tn = (p.N + 63) / 64, tb = (p.B + 63) / 64;
    hipLaunchKernelGGL((int8_stream_kernel<4, 4>), dim3((unsigned)(tn * tb)), dim3(512), 0, stream, p,
                       (int)tn);
  }
  return hipGetLastError();
}

}  // namespace lq
