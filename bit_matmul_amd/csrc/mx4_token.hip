// The 4-bit layer of one token in one launch: every workgroup makes the token's
// codes for itself and multiplies 16 weight rows with them.
//
// int8_token.hip's form: the row is loaded first, then all of the weights are
// on their way to LDS before the codes are made; products as in mx4_few.hip,
// each of the W wavefronts 1024 values of the row and its part of the reduction
// alone, one step of 256 bytes or two. Every lane of a token's column reads the same 16
// bytes of codes, so all 16 columns of a product hold the token's sums, and what the
// wavefronts meet with is 64 bytes each.
//
// In replays of a graph, weights from memory: 8192 -> 10240 10.8 us (4.1 TB/s with
// its launch; in two launches 13.1), with T, which every workgroup makes again, 12.1
// (13.8), with T and a gate 14.4 (14.7); 8192 -> 28672 23.2 (31.1); 14336 -> 4096 8.4 (10.2),
// with a gate 9.5 (11.0; 8 wavefronts of two blocks of 1024 values each took 10.7); 512 -> 1024
// 3.1 (4.7). One workgroup for each compute unit, which makes the codes once and goes on
// from panel to panel through two buffers, was no faster (8192 -> 10240 12.4, with T 13.4;
// 28672 25.6, where this form took 11.2, 14.2 and 22.8): fewer wavefronts have less on
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
  static_assert(S == 1 || S == 2, "steps: 1024 values of the row to a wavefront");
  // (an array for each step: of one the compiler would await all copies before it reads the first)
  __shared__ uint4 stage0[W * kSize];
  __shared__ uint4 stage1[S > 1 ? W * kSize : 1];
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
  Mx4Block<kXBF16, kGate, kScaled, true> in;
  const int col0 = wave * kRowBlock;
  in.load(t, reinterpret_cast<const char*>(t.x), reinterpret_cast<const char*>(t.gate), col0);
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
  if (col0 < W * S * 512) {                        // (S == 1: half of the wavefronts have no values)
    float v[2][8];
    in.values(t, col0, v);
    mx4_transform(t, v);
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const int col = col0 + 512 * j;
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

// One token, a row of at most 16384 values, 8 at a time.
//
// Every 16 outputs make the row again, which a second launch would save. What that
// costs depends on T, the gate and how many workgroups share a compute unit (8 of 4
// wavefronts with one step each, 4 of those with two, 2 of 8). In us for 16 outputs on every
// compute unit, weights from memory: the product of two launches takes kPanel + kValue K, with rows
// of no whole cache lines kRagged more; one launch at most as long without T and gate,
// and with them at least kMake. The second launch itself costs kSaved. Fitted to 1152
// measurements; of them the faster way takes 5120 -> 28672 with T 20.7 us in two launches (22.6 in
// one), 8192 -> 28672 with T 26.2 in one (32.4), 1024 -> 131072 with T and a gate 27.0 in
// two (32.1), with T 20.1 in one (25.7). profiles/mx4_token_times.txt has others; of those
// the rule's choice is 0.2% above the faster way on average, and 15% at most.
//
// Rows of more than 8192 (16 wavefronts, one workgroup to a unit) where every 16 outputs
// have a unit: 11264 -> 4096 with T 8.5 us in one launch, 9.7 in two; -> 8192 15.0 and 14.0. From
// 14336 on without T and gate for any number (16384 -> 28672 44.8 and 54.0), and with both T and a
// gate not below that (12288 -> 1024 9.5 and 9.0).
bool mx4_token_fits(int64_t B, int64_t N, int64_t K, int cus, bool transform, bool gate) {
  // (a launch has fewer than 2^32 threads: 1024 to a workgroup above 8192 inputs)
  if (B != 1 || K % 8 != 0 || K > 16384 || N > (int64_t(1) << (K > 8192 ? 25 : 26))) return false;
  const int64_t panels = (N + 15) / 16;
  if (cus <= 0) cus = 256;
  if (K > 8192) return panels <= cus ? K >= 14336 || !(transform && gate) : K >= 14336 && !transform && !gate;
  if (!transform && !gate) return true;
  constexpr float kPanel = 0.38f, kValue = 0.394f / 1024.0f, kRagged = 0.12f, kSaved = 2.75f;
  // T, a gate, both
  constexpr float kMake[3][3] = {{0.67f, 0.68f, 1.08f}, {0.90f, 0.77f, 1.78f}, {2.95f, 2.83f, 3.58f}};
  const float make = kMake[K > 4096 ? 2 : K > 2048][!transform ? 1 : gate ? 2 : 0];
  const float product = (kPanel + kValue * (float)K) * (K % 256 != 0 ? 1.0f + kRagged : 1.0f);
  return (float)panels / (float)cus * (make - product) <= kSaved;
}

template <bool kXBF16, bool kGate, bool kScaled>
static void enqueue_token(const Mx4Rows& t, const Mx4Gemm& p, hipStream_t stream) {
  const dim3 grid((unsigned)((p.N + 15) / 16));
  if (t.K <= 2048) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 4, 1>), grid, dim3(256), 0, stream, t, p);
  else if (t.K <= 4096) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 4, 2>), grid, dim3(256), 0, stream, t, p);
  else if (t.K <= 8192) hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 8, 2>), grid, dim3(512), 0, stream, t, p);
  else hipLaunchKernelGGL((mx4_token_kernel<kXBF16, kGate, kScaled, 16, 2>), grid, dim3(1024), 0, stream, t, p);
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
