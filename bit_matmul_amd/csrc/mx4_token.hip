// The 4-bit layer of one token in one launch: every workgroup makes the
// token's codes for itself and multiplies 16 kPanels weight rows with them.
//
// int8_token.hip's form: the row is loaded first, then all of the weights are
// on their way to LDS before the codes are made; products as in mx4_few.hip,
// each of the W wavefronts its part of the reduction alone, S steps of 256 bytes at
// most, and they meet at the end. Every lane of a token's column reads the
// same 16 bytes of codes, so all 16 columns of a product hold the token's sums.
#include <type_traits>

#include "lq_mx4_mma.h"
#include "lq_mx4_rows.h"

namespace lq {
namespace {

template <bool kXBF16, bool kGate, bool kScaled, int W, int S, int kPanels>
__global__ __launch_bounds__(64 * W) void mx4_token_kernel(Mx4Rows t, Mx4Gemm p) {
  constexpr int kRows = 16 * kPanels, kCodes = 4 * kPanels;        // copies of 4 rows, 1 KB, each
  constexpr int kCopies = kCodes + kPanels;                        // and of scales, 256 bytes
  constexpr int kSize = kCodes * 64 + kPanels * 16;                // 16-byte units of a wavefront's step
  constexpr int kC = (S + 1) / 2;                                  // blocks of 1024 values to a wavefront
  // (an array for each step: of one the compiler would await all copies before it reads the first)
  __shared__ uint4 stage0[W * kSize];
  __shared__ uint4 stage1[S > 1 ? W * kSize : 1];
  __shared__ uint4 stage2[S > 2 ? W * kSize : 1];
  __shared__ uint4 stage3[S > 3 ? W * kSize : 1];
  __shared__ uint4 codes[W * S * 16];
  __shared__ uint16_t scales[W * S * 8];                           // of a 256: 4 of two blocks each
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int K = (int)p.K, blocks = (K + kMxBlock - 1) / kMxBlock, units = (int)mx4_units(p.K);
  const int all = (blocks + 15) / 16;
  const int s0 = all * wave / W, s1 = all * (wave + 1) / W;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  const int rows = (int)min((int64_t)kRows, p.N - n0);

  // ---- the row's loads, then the weights' copies
  Mx4Block<kXBF16, kGate, kScaled, true> in[kC];
  auto col0 = [&](int i) __attribute__((always_inline)) { return (wave + W * i) * kRowBlock; };
#pragma unroll
  for (int i = 0; i < kC; ++i)
    in[i].load(t, reinterpret_cast<const char*>(t.x), reinterpret_cast<const char*>(t.gate), col0(i));
  const uint8_t* const wbase = p.w + n0 * p.ldw;
  uint32_t off[kCodes];
#pragma unroll
  for (int k = 0; k < kCodes; ++k) off[k] = (uint32_t)min(4 * k + g, rows - 1) * (uint32_t)p.ldw;
  const uint8_t* sbase[kPanels];
#pragma unroll
  for (int k = 0; k < kPanels; ++k)
    sbase[k] = p.w_scale + min(n0 / 16 + k, (p.N - 1) / 16) * ((int64_t)units * 128) + 4 * (lane & 31);
  auto copy_step = [&](int s, uint4* stage) __attribute__((always_inline)) {
    s = min(s, max(s1 - 1, s0));
    uint4* const to = stage + wave * kSize;
#pragma unroll
    for (int k = 0; k < kCodes; ++k) {
      const int blk = 16 * s + (r ^ ((4 * k + g) & 15));
      const uint32_t at = blk < blocks ? 16u * (uint32_t)blk : 0u;     // past K: any bytes, their codes are zero
      __builtin_amdgcn_global_load_lds((const void*)(wbase + (off[k] + at)),
                                       (__attribute__((address_space(3))) void*)(to + k * 64), 16, 0, 0);
    }
    const uint32_t unit = (uint32_t)min(2 * s + (lane >> 5), units - 1);
#pragma unroll
    for (int k = 0; k < kPanels; ++k)
      __builtin_amdgcn_global_load_lds((const void*)(sbase[k] + 128u * unit),
                                       (__attribute__((address_space(3))) void*)(to + kCodes * 64 + 16 * k), 4, 0,
                                       0);
  };
  copy_step(s0, stage0);
  if constexpr (S > 1) copy_step(s0 + 1, stage1);
  if constexpr (S > 2) copy_step(s0 + 2, stage2);
  if constexpr (S > 3) copy_step(s0 + 3, stage3);

  // ---- the token's codes, once the row is there and wherever the copies are.
  // (A wait that another instruction follows: int8_token.hip.)
  constexpr int kVmRow = S * kCopies;
  static_assert(kVmRow < 64, "the counter of loads in flight");
  __builtin_amdgcn_s_waitcnt((kVmRow & 15) | ((kVmRow >> 4) << 14) | (7 << 4) | (15 << 8));
  asm volatile("s_nop 0");
  __builtin_amdgcn_sched_barrier(0);
#pragma unroll
  for (int i = 0; i < kC; ++i) {
    if (col0(i) >= W * S * 512) continue;          // (S == 1: half of the wavefronts have no values)
    float v[2][8];
    in[i].values(t, col0(i), v);
    mx4_transform(t, v);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = col0(i) + 512 * j;
      uint32_t byte;
      const uint32_t w = mx4_piece(v[j], byte);
      reinterpret_cast<uint32_t*>(codes)[col / 8 + lane] = w;
      const int b = (lane >> 2) & 7;
      if ((lane & 3) == 0)
        reinterpret_cast<uint8_t*>(scales)[8 * (col / 256 + (lane >> 5)) + 2 * (b & 3) + (b >> 2)] = (uint8_t)byte;
    }
  }

  // ---- the products
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;
  // All of the codes are written, and the copies stay in flight.
  lds_barrier();
  f32x4 acc[kPanels] = {};
  auto do_step = [&](auto ic, const uint4* stage) __attribute__((always_inline)) {
    constexpr int i0 = decltype(ic)::value;
    constexpr int kVm = (S - 1 - i0) * kCopies;                  // later steps' copies may be in flight
    const int s = s0 + i0;
    if (s >= s1) return;
    i32x4 a[kPanels][4], q[4];
    int sa[kPanels][2], sc[2];
    __builtin_amdgcn_s_waitcnt((kVm & 15) | ((kVm >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("s_nop 0");
    __builtin_amdgcn_sched_barrier(0);
    const uint4* const in = stage + wave * kSize;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int c = 4 * h + g;
#pragma unroll
      for (int i = 0; i < kPanels; ++i) a[i][h] = *reinterpret_cast<const i32x4*>(in + 16 * (16 * i + r) + (c ^ r));
      q[h] = *reinterpret_cast<const i32x4*>(codes + 16 * s + c);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // (a NaN past K times a code of zero would not vanish)
      const int left = blocks - 16 * s - 8 * u;
      const int m = (g < left ? 0xFF : 0) | (4 + g < left ? 0xFF00 : 0);
#pragma unroll
      for (int i = 0; i < kPanels; ++i)
        sa[i][u] = reinterpret_cast<const uint16_t*>(in + kCodes * 64)[128 * i + 64 * u + 4 * r + g] & m;
      sc[u] = scales[4 * (2 * s + u) + g];
    }
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < kPanels; ++i) acc[i] = mfma_mx4<0>(a[i][2 * u], q[2 * u], acc[i], sa[i][u], sc[u]);
#pragma unroll
      for (int i = 0; i < kPanels; ++i) acc[i] = mfma_mx4<1>(a[i][2 * u + 1], q[2 * u + 1], acc[i], sa[i][u], sc[u]);
    }
  };
  do_step(std::integral_constant<int, 0>{}, stage0);
  if constexpr (S > 1) do_step(std::integral_constant<int, 1>{}, stage1);
  if constexpr (S > 2) do_step(std::integral_constant<int, 2>{}, stage2);
  if constexpr (S > 3) do_step(std::integral_constant<int, 3>{}, stage3);
  static_assert(S <= 4, "steps");
  // No copy may still be writing LDS when others write their sums there.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  f32x4* const meet = reinterpret_cast<f32x4*>(stage0);
#pragma unroll
  for (int i = 0; i < kPanels; ++i) meet[(W * i + wave) * 64 + lane] = acc[i];
  __syncthreads();
  const int64_t n = n0 + 16 * wave + 4 * g;
  if (wave >= kPanels || r != 0 || n >= p.N) return;
  float rs[4], bias[4];
  load_mx4_rows(p, n, rs, bias);
  f32x4 sum = meet[W * wave * 64 + lane];
#pragma unroll
  for (int k = 1; k < W; ++k) sum += meet[(W * wave + k) * 64 + lane];
  store_mx4_sums(p, 0, n, rs, bias, sum);
}

}  // namespace

// One token, a row of at most 16384 values, 8 at a time, a product that need not
// split its reduction, and rows for fewer than 2^23 workgroups (a launch has
// fewer than 2^32 threads).
int mx4_token_rows(const Mx4Rows& t, int64_t N, const Mx4Plan& plan) {
  if (t.B != 1 || t.K % 8 != 0 || t.K > 16384 || plan.ksplit != 1) return 0;
  return (N + 15) / 16 < (1 << 23) ? 16 : 0;
}

template <bool kXBF16, bool kGate, bool kScaled>
static void enqueue_token(const Mx4Rows& t, const Mx4Gemm& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16));
  if (t.K <= 2048) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 4, 1, 1>), grid, dim3(256), 0, stream, t, p);
  else if (t.K <= 4096) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 4, 2, 1>), grid, dim3(256), 0, stream, t, p);
  else if (t.K <= 8192) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 8, 2, 1>), grid, dim3(512), 0, stream, t, p);
  else hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 8, 4, 1>), grid, dim3(512), 0, stream, t, p);
}
template <bool kXBF16, bool kGate>
static void enqueue_token(const Mx4Rows& t, const Mx4Gemm& p, hipStream_t stream) {
  if (t.c != nullptr) enqueue_token<kXBF16, kGate, true>(t, p, stream);
  else enqueue_token<kXBF16, kGate, false>(t, p, stream);
}

hipError_t launch_mx4_token(const Mx4Rows& t, const Mx4Gemm& p, int rows, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  if (t.x_bf16) {
    if (t.gate) enqueue_token<true, true>(t, p, stream);
    else enqueue_token<true, false>(t, p, stream);
  } else {
    if (t.gate) enqueue_token<false, true>(t, p, stream);
    else enqueue_token<false, false>(t, p, stream);
  }
  return hipGetLastError();
}

}  // namespace lq
