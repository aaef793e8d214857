// 4-bit product (mx4_gemm.hip gives the formula) of up to 16 tokens: the
// weights are read once, whatever their rate allows.
//
// int8_few.hip's form, byte for byte: a workgroup takes one or two panels of 16
// weight rows, each of its 4 wavefronts a quarter of the reduction, alone,
// in steps of 256 bytes of every row through two stages of LDS of its own, and
// they meet once, at the end. With each step come the scales of 512 values: 256
// bytes of a panel, which lie together in memory, a copy of 4 bytes a lane.
//
// Bound by the weights' stream: 16 tokens 28672 -> 8192 24.2 us (5.2 TB/s, its launch
// included; tiles and a join 28), 4 tokens 23.3, 8 tokens 8192 -> 28672 27.2 (4.6). One
// panel to a workgroup, so that two to four of them share a compute unit and one
// copies while another multiplies; two panels, where 16 tokens' codes would
// be as many bytes as one panel's weights. A third stage was slower (16 tokens 24.5 ->
// 25.1 us, 8 tokens 26.9 -> 29.6): fewer workgroups to a compute unit.
#include <type_traits>

#include "lq_mx4_mma.h"

namespace lq {
namespace {

template <int kTokens, int kPanels>
__global__ __launch_bounds__(256) void mx4_few_kernel(Mx4Gemm p) {
  constexpr int KB = 256, S = 2;
  constexpr int kRows = 16 * kPanels;
  constexpr int kW = kRows / 4, kCodes = kW + kTokens / 4;      // of 4 rows, 1 KB, each
  constexpr int kCopies = kCodes + kPanels + 1;                  // and the scales
  constexpr int kSize = kCodes * 64 + (kPanels + 1) * 16;        // 16-byte units of a wavefront's stage
  __shared__ uint4 stage0[4 * kSize];
  __shared__ uint4 stage1[4 * kSize];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  const int rows = (int)min((int64_t)kRows, p.N - n0), tokens = (int)p.B;
  const int K = (int)p.K, blocks = (K + kMxBlock - 1) / kMxBlock, units = (int)mx4_units(p.K);
  // This wavefront's steps: s0 .. s1 - 1 (none, where the row is that short).
  const int all = (blocks + 15) / 16;
  const int s0 = all * wave / 4, s1 = all * (wave + 1) / 4;

  // Copy k: 4 rows; this lane's row (rows and tokens past the last as the
  // last) and chunk of it.
  const uint8_t* const wbase = p.w + n0 * p.ldw;
  uint32_t off[kCodes];
  int chunk[kCodes];
#pragma unroll
  for (int k = 0; k < kCodes; ++k) {
    const int row = 4 * (k < kW ? k : k - kW) + g;
    off[k] = k < kW ? (uint32_t)min(row, rows - 1) * (uint32_t)p.ldw
                    : (uint32_t)min(row, tokens - 1) * (uint32_t)p.ldq;
    chunk[k] = r ^ (row & 15);
  }
  const uint8_t* sbase[kPanels + 1];
#pragma unroll
  for (int k = 0; k <= kPanels; ++k)
    sbase[k] = (k < kPanels ? p.w_scale + min(n0 / 16 + k, (p.N - 1) / 16) * ((int64_t)units * 128) : p.scale) +
               4 * (lane & 31);
  auto copy_step = [&](int s, uint4* stage) __attribute__((always_inline)) {
    const int at_s = min(s, max(s1 - 1, s0));
#pragma unroll
    for (int k = 0; k < kCodes; ++k) {
      const int blk = 16 * at_s + chunk[k];
      const uint32_t at = blk < blocks ? 16u * (uint32_t)blk : 0u;     // past K: any bytes, masked below
      __builtin_amdgcn_global_load_lds((const void*)((k < kW ? wbase : p.q) + (off[k] + at)),
                                       (__attribute__((address_space(3))) void*)(stage + wave * kSize + k * 64),
                                       16, 0, 0);
    }
    const uint32_t unit = (uint32_t)min(2 * at_s + (lane >> 5), units - 1);
#pragma unroll
    for (int k = 0; k <= kPanels; ++k)
      __builtin_amdgcn_global_load_lds((const void*)(sbase[k] + 128u * unit),
                                       (__attribute__((address_space(3))) void*)(stage + wave * kSize + kCodes * 64 + 16 * k),
                                       4, 0, 0);
  };
  constexpr int kVm = (S - 1) * kCopies;      // the next step's copies may be in flight
  constexpr int kWaitVm = (kVm & 15) | ((kVm >> 4) << 14) | (7 << 4) | (15 << 8);
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;

  // Until the next step's copies at most are in flight. (The s_nop: int8_few.hip.)
  auto wait_step = [&] __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitVm);
    asm volatile("s_nop 0");
    __builtin_amdgcn_sched_barrier(0);
  };
  f32x4 acc[kPanels] = {};
  auto do_step = [&](int s, uint4* stage, bool last) __attribute__((always_inline)) {
    i32x4 a[kPanels][4], c[4];
    int sa[kPanels][2], sc[2];
    wait_step();
    const uint4* const in = stage + wave * kSize;
    const uint16_t* const scales = reinterpret_cast<const uint16_t*>(in + kCodes * 64) + 4 * r + g;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int at = (4 * h + g) ^ r;
#pragma unroll
      for (int i = 0; i < kPanels; ++i) a[i][h] = *reinterpret_cast<const i32x4*>(in + 16 * (16 * i + r) + at);
      c[h] = *reinterpret_cast<const i32x4*>(in + kW * 64 + 16 * (r % kTokens) + ((4 * h + g) ^ (r % kTokens)));
    }
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < kPanels; ++i) sa[i][u] = scales[128 * i + 64 * u];
      sc[u] = scales[128 * kPanels + 64 * u];
    }
    if (last && 2 * KB * (s + 1) > K) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int left = K - 2 * KB * s - 32 * (4 * h + g);        // of these 32 codes, those that count
#pragma unroll
        for (int e = 0; e < 4; ++e) c[h][e] &= (int)mx4_mask(left, e);
      }
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const int left = blocks - 16 * s - 8 * u;
        const int m = (g < left ? 0xFF : 0) | (4 + g < left ? 0xFF00 : 0);
#pragma unroll
        for (int i = 0; i < kPanels; ++i) sa[i][u] &= m;
        sc[u] &= m;
      }
    }
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_sched_barrier(0);
    copy_step(s + S, stage);
#pragma unroll
    for (int u = 0; u < 2; ++u) {
#pragma unroll
      for (int i = 0; i < kPanels; ++i) acc[i] = mfma_mx4<0>(a[i][2 * u], c[2 * u], acc[i], sa[i][u], sc[u]);
#pragma unroll
      for (int i = 0; i < kPanels; ++i) acc[i] = mfma_mx4<1>(a[i][2 * u + 1], c[2 * u + 1], acc[i], sa[i][u], sc[u]);
    }
  };
  // Wavefront i adds up and stores panel i: lane (g, r) holds weight rows
  // 4 g .. 4 g + 3 for token r. Their scales and biases are on their way from here on.
  const int64_t n = n0 + 16 * (wave % kPanels) + 4 * g;
  float rs[4], bias[4];
  load_mx4_rows(p, n, rs, bias);
  __builtin_amdgcn_sched_barrier(0);
  copy_step(s0, stage0);
  copy_step(s0 + 1, stage1);
  int s = s0;
  for (const int whole = min(s1, K / (2 * KB)); s + S <= whole; s += S) {
    do_step(s, stage0, false);
    do_step(s + 1, stage1, false);
  }
  if (s < s1) do_step(s, stage0, true);
  if (s + 1 < s1) do_step(s + 1, stage1, true);

  // No copy may still be writing LDS when others write their sums there.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  f32x4* const meet = reinterpret_cast<f32x4*>(stage0);
#pragma unroll
  for (int i = 0; i < kPanels; ++i) meet[(4 * i + wave) * 64 + lane] = acc[i];
  __syncthreads();
  if (wave >= kPanels || n >= p.N || r >= tokens) return;
  f32x4 sum = meet[4 * wave * 64 + lane];
#pragma unroll
  for (int k = 1; k < 4; ++k) sum += meet[(4 * wave + k) * 64 + lane];
  store_mx4_sums(p, r, n, rs, bias, sum);
}

template <int kTokens, int kPanels>
void enqueue(const Mx4Gemm& p, int tiles, hipStream_t stream) {
  hipLaunchKernelGGL((mx4_few_kernel<kTokens, kPanels>), dim3((unsigned)tiles), dim3(256), 0, stream, p);
}

}  // namespace

hipError_t launch_mx4_few(const Mx4Gemm& p, const Mx4Plan& plan, hipStream_t stream) {
  switch (plan.tokens * 2 + plan.rows / 32) {
    case 8: enqueue<4, 1>(p, plan.tiles, stream); break;
    case 16: enqueue<8, 1>(p, plan.tiles, stream); break;
    case 32: enqueue<16, 1>(p, plan.tiles, stream); break;
    case 33: enqueue<16, 2>(p, plan.tiles, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace lq
