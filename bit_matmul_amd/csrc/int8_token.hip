// The 8-bit layer of one token in one launch: every workgroup makes the
// token's codes for itself and multiplies 32 weight rows with them.
//
// Codes as in quant_rows.hip, of the whole row (16 values in each thread's
// registers), into LDS; products as in int8_gemm.hip, steps of
// 256 bytes of 32 rows through four stages. Wavefront (wn, wk) takes panel wn
// and half wk of each step, and the two halves meet in LDS. Every lane of a
// token's column reads the same 16 codes, so all 16 columns of a product hold
// the token's sums.
//
// The weights' stages are filled while the codes are made: the row is loaded
// first (loads return in order, and its wait is then not the weights').
//
// Taken for rows of up to 4096 values. Every workgroup does the arithmetic of
// the row, which the others' streams cover while it is short: against two
// launches 512 x 512 takes 3.9 us for 6.0, 4096 x 2048 6.1 for 8.4, 28672 x
// 4096 28.0 for 31.4; but of 8192 values 8192 outputs 20.5 for 22.4 and 28672
// outputs 56.3 for 50.0.
#include <type_traits>

#include "lq_int8.h"
#include "lq_rows.h"

namespace lq {
namespace {

template <bool kXBF16>
__global__ __launch_bounds__(256, 2) void int8_token_kernel(QuantRows t, Int8Gemm p) {
  constexpr int C = 1, S = 4, KB = 256;
  __shared__ uint4 stage0[512];
  __shared__ uint4 stage1[512];
  __shared__ uint4 stage2[512];
  __shared__ uint4 stage3[512];
  __shared__ uint4 codes[C * 256];            // a block of 1024 for each wavefront
  __shared__ float red[kRowMaxWaves];
  __shared__ i32x4 meet[2 * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int K = (int)p.K, K16 = (K + 15) & ~15;
  const int steps = (K16 + KB - 1) / KB;
  const int64_t n0 = (int64_t)blockIdx.x * 32;
  const int rows = (int)min((int64_t)32, p.N - n0);

  // ---- the row's loads, then the first stages' copies
  const bool whole = row_whole<C>(K);
  RowPiece<kXBF16> x[C][2];
  auto load = [&](auto wholec) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < C; ++i)
#pragma unroll
      for (int j = 0; j < 2; ++j) load_piece(x[i][j], t.x, row_col(i, j), K, decltype(wholec)::value);
  };
  if (whole) load(std::true_type{});
  else load(std::false_type{});

  // Copy k (0, 1) of a wavefront: 4 rows; this lane's row and chunk.
  const int row = 4 * wave + (lane >> 4);
  const int chunk = (lane & 15) ^ row;
  const int8_t* const wbase = p.w + n0 * p.ldw;
  uint32_t off[2];
#pragma unroll
  for (int k = 0; k < 2; ++k) off[k] = (uint32_t)min(16 * k + row, rows - 1) * (uint32_t)p.ldw;
  auto copy_step = [&](int s, uint4* dst) __attribute__((always_inline)) {
    const uint32_t c = (uint32_t)KB * (uint32_t)min(s, steps - 1) + 16u * (uint32_t)chunk;
    const uint32_t at = c < (uint32_t)K16 ? c : 0u;      // past K: any bytes, their codes are zero
#pragma unroll
    for (int k = 0; k < 2; ++k)
      __builtin_amdgcn_global_load_lds((const void*)(wbase + (off[k] + at)),
                                       (__attribute__((address_space(3))) void*)(dst + (wave + 4 * k) * 64), 16,
                                       0, 0);
  };
  copy_step(0, stage0);
  copy_step(1, stage1);
  copy_step(2, stage2);

  // ---- the token's codes
  float v[C][2][8];
  float m = 0.0f;
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j) x[i][j].get(v[i][j]);
  if (t.c != nullptr) {
#pragma unroll
    for (int i = 0; i < C; ++i) {
      RowPiece<false> c[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) load_piece(c[j], t.c, row_col(i, j), K, whole);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        float a[8];
        c[j].get(a);
#pragma unroll
        for (int k = 0; k < 8; ++k) v[i][j][k] *= a[k];
      }
    }
  }
  if (t.lhb > 0) {
#pragma unroll
    for (int i = 0; i < C; ++i) fwht_block(v[i], t.lhb);
  }
#pragma unroll
  for (int i = 0; i < C; ++i)
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(v[i][j][k]));
  m = row_reduce<MaxBits>(m, red);
  const RowCoder coder(m);
#pragma unroll
  for (int i = 0; i < C; ++i) {
    uint2 w[2] = {coder.codes(v[i][0]), coder.codes(v[i][1])};
    if (t.lhb > 7) fwht_order(w, t.lhb);
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<uint2*>(reinterpret_cast<int8_t*>(codes) + row_col(i, j) + row_lane8()) = w[j];
  }

  // ---- the products
  constexpr int kWaitVm = (S - 2) * 2 | (7 << 4) | (15 << 8);    // the copies of two steps may be in flight
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;
  const int wn = wave & 1, wk = wave >> 1;
  i32x4 acc = {0, 0, 0, 0};
  auto stage_c = [&](auto ic) __attribute__((always_inline)) -> uint4* {
    constexpr int i = decltype(ic)::value % S;
    if constexpr (i == 0) return stage0;
    else if constexpr (i == 1) return stage1;
    else if constexpr (i == 2) return stage2;
    else return stage3;
  };
  // Passing the barrier, the step's stage is full and the step before it (and
  // the codes) are done with: its stage takes the copies of three steps on.
  auto do_step = [&](auto sc, int s) __attribute__((always_inline)) {
    constexpr int su = decltype(sc)::value;
    const uint4* const cur = stage_c(std::integral_constant<int, su>{});
    __builtin_amdgcn_s_waitcnt(kWaitVm);
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_s_barrier();
    copy_step(s + 3, stage_c(std::integral_constant<int, su + 3>{}));
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const int c = 4 * (2 * wk + h) + g;
      const i32x4 a = *reinterpret_cast<const i32x4*>(cur + wn * 256 + 16 * r + (c ^ r));
      const i32x4 q = *reinterpret_cast<const i32x4*>(codes + 16 * s + c);
      acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, q, acc, 0, 0, 0);
    }
  };
  for (int s = 0;;) {
    do_step(std::integral_constant<int, 0>{}, s);
    if (++s == steps) break;
    do_step(std::integral_constant<int, 1>{}, s);
    if (++s == steps) break;
    do_step(std::integral_constant<int, 2>{}, s);
    if (++s == steps) break;
    do_step(std::integral_constant<int, 3>{}, s);
    if (++s == steps) break;
  }
  // No copy may still be writing LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(0);
  if (wk == 1) meet[wn * 64 + lane] = acc;
  __syncthreads();
  const int64_t n = n0 + 16 * wn + 4 * g;
  if (wk == 1 || r != 0 || n >= p.N) return;
  acc += meet[wn * 64 + lane];
  float rs[4], bias[4];
  load_int8_rows(p, n, rs, bias);
  store_int8_sums(p, 0, n, coder.scale(t.norm), rs, bias, acc);
}

}  // namespace

// One token, no gate, a short row, and a product that need not split its
// reduction to fill the device (that is a launch more, as this is one less).
bool int8_token_applies(const QuantRows& t, const Int8Plan& plan) {
  return t.B == 1 && t.gate == nullptr && t.K <= 4 * kRowBlock && plan.ksplit == 1;
}

hipError_t launch_int8_token(const QuantRows& t, const Int8Gemm& p, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  const dim3 grid((unsigned)((p.N + 31) / 32));
  if (t.x_bf16) hipLaunchKernelGGL((int8_token_kernel<true>), grid, dim3(256), 0, stream, t, p);
  else hipLaunchKernelGGL((int8_token_kernel<false>), grid, dim3(256), 0, stream, t, p);
  return hipGetLastError();
}

}  // namespace lq
