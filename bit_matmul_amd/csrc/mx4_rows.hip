// Microscaled 4-bit rows (include/lq.h gives the format) of v = T (act(gate)
// .* x): the rows and weights of the 4-bit product.
//
// A block's scale needs its own 32 values alone, T its own 1024, so no
// wavefront waits for another: each takes 1024 values of a row (lq_rows.h:
// a lane 8 values of each half), a block is four lanes, and its maximum two
// lane exchanges. The conversion is the hardware's: v_cvt_scalef32_pk_fp4_f32
// divides by the power of two, which is exact, and rounds to the nearest value,
// ties to the even code, what is above 6 to 6.
//
// Bound by the bytes, from memory: 2048 x 28672 bf16 32 us (4.7 TB/s), with a gate 58 (4.5);
// with T 2048 x 8192 15.7 us, where the same without T takes 10.5: the butterflies and the
// channel scales, read for every row. 16 rows to a workgroup, whose scales lie together,
// were no faster, nor was a cheaper sigmoid.
#include "lq_mx4_rows.h"

namespace lq {
namespace {

template <bool kXBF16, bool kGate, bool kScaled, bool kEven>
__global__ __launch_bounds__(256) void mx4_rows_kernel(Mx4Rows p) {
  const int64_t b = (int64_t)blockIdx.z * gridDim.x + blockIdx.x;
  const int K = (int)p.K;
  const int col0 = ((int)blockIdx.y * ((int)blockDim.x >> 6) + wave_id()) * kRowBlock;
  if (b >= p.B || col0 >= K) return;
  const int lane = threadIdx.x & 63;
  const char* const xrow = reinterpret_cast<const char*>(p.x) + b * p.ldx * (kXBF16 ? 2 : 4);
  const char* const grow = reinterpret_cast<const char*>(p.gate) + b * p.ldg * (kXBF16 ? 2 : 4);
  Mx4Block<kXBF16, kGate, kScaled, kEven> in;
  in.load(p, xrow, grow, col0);
  float v[2][8];
  in.values(p, col0, v);
  mx4_transform(p, v);
  const int units = (int)mx4_units(p.K), bytes = (int)mx4_row_bytes(p.K);
#pragma unroll
  for (int j = 0; j < 2; ++j) {
    uint32_t byte;
    const uint32_t w = mx4_piece(v[j], byte);
    const int at = (col0 + 512 * j) / 2 + 4 * lane;
    if (at < bytes) *reinterpret_cast<uint32_t*>(p.q + b * p.ldq + at) = w;
    // the first lane of a block: block i of unit u
    const int u = (col0 + 512 * j) / kMxUnit + (lane >> 5), i = (lane >> 2) & 7;
    if ((lane & 3) == 0 && u < units)
      p.scale[((b >> 4) * units + u) * 128 + 8 * (b & 15) + 2 * (i & 3) + (i >> 2)] = (uint8_t)byte;
  }
}

constexpr int64_t kGridRows = 1 << 22;

template <bool kScaled, bool kEven>
void enqueue(const Mx4Rows& p, dim3 grid, dim3 block, hipStream_t stream) {
  if (p.x_bf16) {
    if (p.gate) hipLaunchKernelGGL((mx4_rows_kernel<true, true, kScaled, kEven>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((mx4_rows_kernel<true, false, kScaled, kEven>), grid, block, 0, stream, p);
  } else {
    if (p.gate) hipLaunchKernelGGL((mx4_rows_kernel<false, true, kScaled, kEven>), grid, block, 0, stream, p);
    else hipLaunchKernelGGL((mx4_rows_kernel<false, false, kScaled, kEven>), grid, block, 0, stream, p);
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
  const bool even = p.K % 8 == 0;
  if (p.c != nullptr) {
    if (even) enqueue<true, true>(p, grid, block, stream);
    else enqueue<true, false>(p, grid, block, stream);
  } else {
    if (even) enqueue<false, true>(p, grid, block, stream);
    else enqueue<false, false>(p, grid, block, stream);
  }
  return hipGetLastError();
}

}  // namespace lq
