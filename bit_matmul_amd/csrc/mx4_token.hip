// The 4-bit layer of one token in one launch: every workgroup makes the token's
// codes for itself and multiplies 16 weight rows with them.
//
// int8_token.hip's form: the row is loaded first, then all of the weights are
// on their way to LDS before the codes are made; products as in mx4_few.hip,
// each of the W wavefronts its part of the reduction alone, S steps of 256 bytes
// at most. Every lane of a token's column reads the same 16 bytes of codes, so
// all 16 columns of a product hold the token's sums, and what the wavefronts meet
// with is 64 bytes each.
//
// In replays of a graph, weights from memory: 8192 -> 10240 11.2 us (4.0 TB/s with
// its launch; in two launches 13.9), with T, which every workgroup makes again, 14.2
// (14.5); 8192 -> 28672 22.8 (26.0; 5.5 TB/s); 4096 -> 14336 7.7; 14336 -> 4096 8.7, with a
// gate 10.9; 512 -> 512 2.4 (4.3). One workgroup for each compute unit, which
// makes the codes once and goes on from panel to panel through two buffers, was no
// faster (8192 -> 10240 12.4, with T 13.4; 28672 25.6): fewer wavefronts have less on
// their way.
#include <type_traits>

#include "lq_mx4_mma.h"
#include "lq_mx4_rows.h"

namespace lq {
namespace {

template <bool kXBF16, bool kGate, bool kScaled, int W, int S>
__global__ __launch_bounds__(64 * W) void mx4_token_kernel(Mx4Rows t, Mx4Gemm p) {
  constexpr int kCopies = 4 + 1;                                   // of codes, 4 rows, 1 KB, each, and of scales, 256 bytes
  constexpr int kSize = 4 * 64 + 16;                               // 16-byte units of a wavefront's step
  constexpr int kC = (S + 1) / 2;                                  // blocks of 1024 values to a wavefront
  // (an array for each step: of one the compiler would await all copies before it reads the first)
  __shared__ uint4 stage0[W * kSize];
  __shared__ uint4 stage1[S > 1 ? W * kSize : 1];
  __shared__ uint4 stage2[S > 2 ? W * kSize : 1];
  __shared__ uint4 stage3[S > 3 ? W * kSize : 1];
  __shared__ uint4 codes[W * S * 16];
  __shared__ uint16_t scales[W * S * 8];                           // of a 256: 4 of two blocks each
  __shared__ __attribute__((aligned(16))) float meet[W * 16];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int K = (int)p.K, blocks = (K + kMxBlock - 1) / kMxBlock, units = (int)mx4_units(p.K);
  const int all = (blocks + 15) / 16;
  const int s0 = all * wave / W, s1 = all * (wave + 1) / W;
  const int64_t n0 = (int64_t)blockIdx.x * 16;
  const int rows = (int)min((int64_t)16, p.N - n0);

  // ---- the row's loads, then the weights' copies, then this thread's output's scale and bias
  Mx4Block<kXBF16, kGate, kScaled, true> in[kC];
  auto col0 = [&](int i) __attribute__((always_inline)) { return (wave + W * i) * kRowBlock; };
#pragma unroll
  for (int i = 0; i < kC; ++i)
    in[i].load(t, reinterpret_cast<const char*>(t.x), reinterpret_cast<const char*>(t.gate), col0(i));
  // (Loads and copies are counted below: in this order.)
  __builtin_amdgcn_sched_barrier(0);
  const uint8_t* const wbase = p.w + n0 * p.ldw;
  const uint8_t* const sbase = p.w_scale + (int64_t)blockIdx.x * ((int64_t)units * 128) + 4 * (lane & 31);
  auto copy_step = [&](int i, uint4* stage) __attribute__((always_inline)) {
    const int s = min(s0 + i, max(s1 - 1, s0));
    uint4* const to = stage + wave * kSize;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const int blk = 16 * s + (r ^ (4 * k + g));
      const uint32_t at = blk < blocks ? 16u * (uint32_t)blk : 0u;     // past K: any bytes, their codes are zero
      __builtin_amdgcn_global_load_lds((const void*)(wbase + ((uint32_t)min(4 * k + g, rows - 1) * (uint32_t)p.ldw + at)),
                                       (__attribute__((address_space(3))) void*)(to + k * 64), 16, 0, 0);
    }
    __builtin_amdgcn_global_load_lds((const void*)(sbase + 128u * (uint32_t)min(2 * s + (lane >> 5), units - 1)),
                                     (__attribute__((address_space(3))) void*)(to + 256), 4, 0, 0);
  };
  copy_step(0, stage0);
  if constexpr (S > 1) copy_step(1, stage1);
  if constexpr (S > 2) copy_step(2, stage2);
  if constexpr (S > 3) copy_step(3, stage3);
  // (Loads return in order: before the row, these, from memory, would hold it up.
  // Two loads in every thread, of any bytes where there are none, so that all count alike.)
  const int64_t n = n0 + threadIdx.x;
  const bool mine = (int)threadIdx.x < rows;
  const float* const none = reinterpret_cast<const float*>(p.w_scale);
  const float rs_ = *(p.row_scale != nullptr ? p.row_scale + (mine ? n : 0) : none);
  const float bias_ = *(p.bias != nullptr ? p.bias + (mine ? n : 0) : none);
  __builtin_amdgcn_sched_barrier(0);

  // ---- the token's codes, once the row is there and wherever the copies are.
  // (A wait that another instruction follows: int8_token.hip.)
  constexpr int kVmRow = S * kCopies + 2;
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
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  auto do_step = [&](auto ic, const uint4* stage) __attribute__((always_inline)) {
    constexpr int i0 = decltype(ic)::value;
    constexpr int kVm = (S - 1 - i0) * kCopies + 2;              // later steps' copies may be in flight
    const int s = s0 + i0;
    i32x4 a[4], q[4];
    int sa[2], sc[2];
    __builtin_amdgcn_s_waitcnt((kVm & 15) | ((kVm >> 4) << 14) | (7 << 4) | (15 << 8));
    asm volatile("s_nop 0");
    __builtin_amdgcn_sched_barrier(0);
    const uint4* const in = stage + wave * kSize;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int c = 4 * h + g;
      a[h] = *reinterpret_cast<const i32x4*>(in + 16 * r + (c ^ r));
      q[h] = *reinterpret_cast<const i32x4*>(codes + 16 * s + c);
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      // Past K a NaN times a code of zero would not vanish; a step that is
      // another wavefront's: both scales 2^-127, whose product is nothing.
      const int left = s < s1 ? blocks - 16 * s - 8 * u : 0;
      const int m = (g < left ? 0xFF : 0) | (4 + g < left ? 0xFF00 : 0);
      sa[u] = reinterpret_cast<const uint16_t*>(in + 256)[64 * u + 4 * r + g] & m;
      sc[u] = scales[4 * (2 * s + u) + g] & m;
    }
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      acc = mfma_mx4<0>(a[2 * u], q[2 * u], acc, sa[u], sc[u]);
      acc = mfma_mx4<1>(a[2 * u + 1], q[2 * u + 1], acc, sa[u], sc[u]);
    }
  };
  do_step(std::integral_constant<int, 0>{}, stage0);
  if constexpr (S > 1) do_step(std::integral_constant<int, 1>{}, stage1);
  if constexpr (S > 2) do_step(std::integral_constant<int, 2>{}, stage2);
  if constexpr (S > 3) do_step(std::integral_constant<int, 3>{}, stage3);
  static_assert(S <= 4, "steps");
  // (here, by all lanes: the compiler moved the products, and the masks of their
  // scales with them, behind the test below)
  asm volatile("" : "+v"(acc));
  if (r == 0) *reinterpret_cast<f32x4*>(meet + wave * 16 + 4 * g) = acc;
  __syncthreads();
  if (!mine) return;
  const float rs = p.row_scale != nullptr ? rs_ : 1.0f, bias = p.bias != nullptr ? bias_ : 0.0f;
  float sum = meet[threadIdx.x];
#pragma unroll
  for (int k = 1; k < W; ++k) sum += meet[16 * k + threadIdx.x];
  const float v = fmaf(sum, rs, bias);
  if (p.y_bf16) reinterpret_cast<uint16_t*>(p.y)[n] = (uint16_t)f32_to_bf16_bits(v);
  else reinterpret_cast<float*>(p.y)[n] = v;
}

}  // namespace

// One token, a row of at most 16384 values, 8 at a time, and of more than 8192
// only where every 16 rows have a compute unit: LDS holds no more of those, and the row would be
// made again for each (14336 -> 4096 with a gate 10.9 us, in two launches 11.1).
bool mx4_token_fits(int64_t B, int64_t N, int64_t K, int cus) {
  if (B != 1 || K % 8 != 0 || N > (int64_t(1) << 26)) return false;
  return K <= 8192 || (K <= 16384 && (N + 15) / 16 <= (cus > 0 ? cus : 256));
}

template <bool kXBF16, bool kGate, bool kScaled>
static void enqueue_token(const Mx4Rows& t, const Mx4Gemm& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16));
  if (t.K <= 2048) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 4, 1>), grid, dim3(256), 0, stream, t, p);
  else if (t.K <= 4096) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 4, 2>), grid, dim3(256), 0, stream, t, p);
  else if (t.K <= 8192) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 8, 2>), grid, dim3(512), 0, stream, t, p);
  else hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 8, 4>), grid, dim3(512), 0, stream, t, p);
}
template <bool kXBF16, bool kGate>
static void enqueue_token(const Mx4Rows& t, const Mx4Gemm& p, hipStream_t stream) {
  if (t.c != nullptr) enqueue_token<kXBF16, kGate, true>(t, p, stream);
  else enqueue_token<kXBF16, kGate, false>(t, p, stream);
}

hipError_t launch_mx4_token(const Mx4Rows& t, const Mx4Gemm& p, hipStream_t stream) {
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
