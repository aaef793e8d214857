// The 8-bit layer of one token in one launch: every workgroup makes the
// token's codes for itself and multiplies 16 kPanels weight rows with them.
//
// Codes as in quant_rows.hip, of the whole row (16 values in each thread's
// registers), into LDS; products as in int8_few.hip: each of the 4 wavefronts
// takes its quarter of the reduction alone, S steps of 256 bytes at most, and
// they meet at the end. All of the weights are on their way to LDS before the
// codes are made; the row is loaded first (loads return in order), and nothing
// on the way to the codes waits for the weights. Every lane of a token's
// column reads the same 16 codes, so all 16 columns of a product hold the
// token's sums.
//
// Taken for rows of up to 4096 values. Every workgroup does the arithmetic of
// the row, which the others' streams cover while it is short: against two
// launches 512 x 512 takes 3.8 us for 5.1, 4096 x 2048 4.6 for 6.5, 8192 x 4096
// 9.0 for 11.8, 28672 x 4096 23.6 for 29.5. A longer row would be twice the
// arithmetic and twice the LDS. Many rows of few values are mostly that
// arithmetic, the transform's above all: there two panels to a workgroup halve
// it (with T 16384 x 1024 7.3 -> 6.3 us, 60000 x 512 17.7 -> 13.4; without T
// 60000 x 512 12.1 -> 11.1, but 28672 x 512 6.2 -> 6.5; 28672 x 2048 with T
// 14.7 either way).
#include <type_traits>

#include "lq_int8.h"
#include "lq_rows.h"

namespace lq {
namespace {

template <bool kXBF16, int S, int kPanels>
__global__ __launch_bounds__(256) void int8_token_kernel(QuantRows t, Int8Gemm p) {
  constexpr int KB = 256;
  constexpr int kRows = 16 * kPanels, kCopies = 4 * kPanels;       // of 4 rows, 1 KB, each
  __shared__ uint4 stage0[4 * kCopies * 64];
  __shared__ uint4 stage1[S > 1 ? 4 * kCopies * 64 : 1];
  __shared__ uint4 stage2[S > 2 ? 4 * kCopies * 64 : 1];
  __shared__ uint4 stage3[S > 3 ? 4 * kCopies * 64 : 1];
  __shared__ uint4 codes[256];                // a block of 1024 for each wavefront
  __shared__ float red[kRowMaxWaves];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int K = (int)p.K, K16 = (K + 15) & ~15;
  const int all = (K + KB - 1) / KB;
  const int s0 = all * wave / 4, s1 = all * (wave + 1) / 4;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  const int rows = (int)min((int64_t)kRows, p.N - n0);

  // ---- the row's loads, then the first stages' copies
  const bool whole = row_whole<1>(K);
  RowPiece<kXBF16> x[2];
  RowPiece<false> c[2];
  auto load = [&](auto wholec) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < 2; ++j) load_piece(x[j], t.x, row_col(0, j), K, decltype(wholec)::value);
    if (t.c != nullptr) {
#pragma unroll
      for (int j = 0; j < 2; ++j) load_piece(c[j], t.c, row_col(0, j), K, decltype(wholec)::value);
    }
  };
  if (whole) load(std::true_type{});
  else load(std::false_type{});

  // Copy k: 4 rows; this lane's row and chunk of it.
  const int8_t* const wbase = p.w + n0 * p.ldw;
  uint32_t off[kCopies], chunk[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    off[k] = (uint32_t)min(4 * k + g, rows - 1) * (uint32_t)p.ldw;
    chunk[k] = 16u * (uint32_t)(r ^ ((4 * k + g) & 15));
  }
  auto copy_step = [&](int s, uint4* stage) __attribute__((always_inline)) {
    const uint32_t base = (uint32_t)KB * (uint32_t)min(s, max(s1 - 1, s0));
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const uint32_t c = base + chunk[k], at = c < (uint32_t)K16 ? c : 0u;   // past K: any bytes, their codes are zero
      __builtin_amdgcn_global_load_lds((const void*)(wbase + (off[k] + at)),
                                       (__attribute__((address_space(3))) void*)(stage + (wave * kCopies + k) * 64),
                                       16, 0, 0);
    }
  };
  copy_step(s0, stage0);
  if constexpr (S > 1) copy_step(s0 + 1, stage1);
  if constexpr (S > 2) copy_step(s0 + 2, stage2);
  if constexpr (S > 3) copy_step(s0 + 3, stage3);

  // ---- the token's codes, once the row is there and wherever the copies are.
  // (A wait that another instruction follows: the compiler's own would be for
  // the copies too.)
  constexpr int kVmRow = S * kCopies;
  static_assert(kVmRow < 64, "the counter of loads in flight");
  __builtin_amdgcn_s_waitcnt((kVmRow & 15) | ((kVmRow >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("s_nop 0");
  __builtin_amdgcn_sched_barrier(0);
  float v[2][8];
  float m = 0.0f;
#pragma unroll
  for (int j = 0; j < 2; ++j) x[j].get(v[j]);
  if (t.c != nullptr) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      float a[8];
      c[j].get(a);
#pragma unroll
      for (int k = 0; k < 8; ++k) v[j][k] *= a[k];
    }
  }
  if (t.lhb > 0) fwht_block(v, t.lhb);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int k = 0; k < 8; ++k) m = MaxBits::of(m, fabsf(v[j][k]));
  m = row_reduce<MaxBits>(m, red);
  const RowCoder coder(m);
  uint2 w[2] = {coder.codes(v[0]), coder.codes(v[1])};
  if (t.lhb > 7) fwht_order(w, t.lhb);
#pragma unroll
  for (int j = 0; j < 2; ++j)
    *reinterpret_cast<uint2*>(reinterpret_cast<int8_t*>(codes) + row_col(0, j) + row_lane8()) = w[j];

  // ---- the products
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;
  // All of the codes are written, and the copies stay in flight.
  lds_barrier();
  i32x4 acc[kPanels] = {};
  auto do_step = [&](auto ic, uint4* stage) __attribute__((always_inline)) {
    constexpr int i0 = decltype(ic)::value;
    constexpr int kVm = (S - 1 - i0) * kCopies;                  // later steps' copies may be in flight
    const int s = s0 + i0;
    if (s >= s1) return;
    i32x4 a[kPanels][4], q[4];
    __builtin_amdgcn_s_waitcnt((kVm & 15) | ((kVm >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("s_nop 0");
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int c = 4 * h + g;
#pragma unroll
      for (int i = 0; i < kPanels; ++i)
        a[i][h] = *reinterpret_cast<const i32x4*>(stage + wave * kCopies * 64 + 16 * (16 * i + r) + (c ^ r));
      q[h] = *reinterpret_cast<const i32x4*>(codes + 16 * s + c);
    }
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int i = 0; i < kPanels; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i][h], q[h], acc[i], 0, 0, 0);
  };
  do_step(std::integral_constant<int, 0>{}, stage0);
  if constexpr (S > 1) do_step(std::integral_constant<int, 1>{}, stage1);
  if constexpr (S > 2) do_step(std::integral_constant<int, 2>{}, stage2);
  if constexpr (S > 3) do_step(std::integral_constant<int, 3>{}, stage3);
  // No copy may still be writing LDS when others write their sums there.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  i32x4* const meet = reinterpret_cast<i32x4*>(stage0);
#pragma unroll
  for (int i = 0; i < kPanels; ++i) meet[(4 * i + wave) * 64 + lane] = acc[i];
  __syncthreads();
  const int64_t n = n0 + 16 * wave + 4 * g;
  if (wave >= kPanels || r != 0 || n >= p.N) return;
  i32x4 sum = meet[4 * wave * 64 + lane];
#pragma unroll
  for (int k = 1; k < 4; ++k) sum += meet[(4 * wave + k) * 64 + lane];
  float rs[4], bias[4];
  load_int8_rows(p, n, rs, bias);
  store_int8_sums(p, 0, n, coder.scale(t.norm), rs, bias, sum);
}

}  // namespace

// One token, no gate, a short row, a product that need not split its
// reduction to fill the device (that is a launch more, as this is one less),
// and rows for fewer than 2^24 workgroups of 256 (a launch has fewer than 2^32
// threads; the tiles of more rows take more of them).
int int8_token_rows(const QuantRows& t, int64_t N, const Int8Plan& plan) {
  if (t.B != 1 || t.gate != nullptr || t.K > 4 * kRowBlock || plan.ksplit != 1) return 0;
  const int64_t many = t.lhb > 0 ? 8192 : 32768;      // rows from which on two panels pay (see the top)
  const int rows = t.K <= kRowBlock && N > many ? 32 : 16;
  return (N + rows - 1) / rows < (1 << 24) ? rows : 0;
}

template <int S, int kPanels>
static void enqueue_token(const QuantRows& t, const Int8Gemm& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 16 * kPanels - 1) / (16 * kPanels)));
  if (t.x_bf16) hipLaunchKernelGGL((int8_token_kernel<true, S, kPanels>), grid, dim3(256), 0, stream, t, p);
  else hipLaunchKernelGGL((int8_token_kernel<false, S, kPanels>), grid, dim3(256), 0, stream, t, p);
}

hipError_t launch_int8_token(const QuantRows& t, const Int8Gemm& p, int rows, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  if (rows == 32) enqueue_token<1, 2>(t, p, stream);
  else if (t.K <= kRowBlock) enqueue_token<1, 1>(t, p, stream);
  else if (t.K <= 2 * kRowBlock) enqueue_token<2, 1>(t, p, stream);
  else enqueue_token<4, 1>(t, p, stream);
  return hipGetLastError();
}

}  // namespace lq
