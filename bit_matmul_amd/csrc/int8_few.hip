// 8-bit product (int8_gemm.hip gives the formula) of up to 16 tokens: the
// weights are read once, whatever their rate allows.
//
// A workgroup takes one or two panels of 16 weight rows; each of its 4
// wavefronts a quarter of the reduction, alone: it copies its own weights and
// codes to LDS (global_load_lds), in steps of 256 bytes of every row through
// two stages, waits for its own copies only and meets the others once, at the
// end, in LDS. Without a barrier in the loop the wavefronts drift apart and
// their loads never stop together, and with 16 rows to a workgroup there are
// enough of them that the reduction need not be split over a second launch.
// Against tiles of 32 rows and 32 tokens with a barrier in each step and a
// join (one token, product alone): 4096 x 14336 16.6 -> 12.6 us, 10240 x 8192
// 22.7 -> 18.9, 8192 x 28672 49.0 -> 43.5 (5.4 TB/s), 1000 x 2050 5.8 -> 3.8.
// Three or four stages, fewer workgroups on a compute unit, gave nothing
// (5125 x 4099 8.0 -> 8.3 and 8.6 us).
//
// Codes are copied for kTokens tokens only, 4, 8 or 16: columns of the
// product that belong to none hold whatever was in LDS and are not stored.
// Every 16 rows read the codes of their quarter again: at 16 tokens as many
// bytes as weights, which is what two panels halve (8192 x 28672 48.9 -> 45.0
// us) where their workgroups, fewer and larger, still fill the device evenly
// (10240 x 8192 21.8 -> 24.2).
//
// Row r of a step keeps its 16-byte chunk c at 16 r + (c ^ (r & 15)), as in
// int8_gemm.hip: no bank conflicts, whole lines copied.
#include <type_traits>

#include "lq_int8.h"

namespace lq {
namespace {

template <int kTokens, int kPanels>
__global__ __launch_bounds__(256) void int8_few_kernel(Int8Gemm p) {
  constexpr int KB = 256, S = 2;
  constexpr int kRows = 16 * kPanels;
  constexpr int kW = kRows / 4, kCopies = kW + kTokens / 4;     // of 4 rows, 1 KB, each
  constexpr int kSize = kCopies * 64;                            // 16-byte units of a wavefront's stage
  __shared__ uint4 stage0[4 * kSize];
  __shared__ uint4 stage1[4 * kSize];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int64_t n0 = (int64_t)blockIdx.x * kRows;
  const int rows = (int)min((int64_t)kRows, p.N - n0), tokens = (int)p.B;
  const int K = (int)p.K, K16 = (K + 15) & ~15;
  // This wavefront's steps: s0 .. s1 - 1 (none, where the row is that short).
  const int all = (K + KB - 1) / KB;
  const int s0 = all * wave / 4, s1 = all * (wave + 1) / 4;

  // Copy k: 4 rows; this lane's row (rows and tokens past the last as the
  // last) and chunk of it.
  const int8_t* const wbase = p.w + n0 * p.ldw;
  uint32_t off[kCopies], chunk[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    const int row = 4 * (k < kW ? k : k - kW) + g;
    off[k] = k < kW ? (uint32_t)min(row, rows - 1) * (uint32_t)p.ldw
                    : (uint32_t)min(row, tokens - 1) * (uint32_t)p.ldq;
    chunk[k] = 16u * (uint32_t)(r ^ (row & 15));
  }
  auto copy_step = [&](int s, uint4* stage) __attribute__((always_inline)) {
    const uint32_t base = (uint32_t)KB * (uint32_t)min(s, max(s1 - 1, s0));
#pragma unroll
    for (int k = 0; k < kCopies; ++k) {
      const uint32_t c = base + chunk[k], at = c < (uint32_t)K16 ? c : 0u;   // past K: any bytes, masked below
      __builtin_amdgcn_global_load_lds((const void*)((k < kW ? wbase : p.q) + (off[k] + at)),
                                       (__attribute__((address_space(3))) void*)(stage + wave * kSize + k * 64),
                                       16, 0, 0);
    }
  };
  constexpr int kWaitVm = (S - 1) * kCopies | (7 << 4) | (15 << 8);    // the next step's copies may be in flight
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;
  static_assert((S - 1) * kCopies < 16, "the counter's low bits");

  // Until the next step's copies at most are in flight. (The compiler waits
  // for copies of its own accord before it reads where they went, and then
  // for all of them. Only a wait that is followed by another instruction
  // counts as one already done: hence the s_nop.)
  auto wait_step = [&] __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(kWaitVm);
    asm volatile("s_nop 0");
    __builtin_amdgcn_sched_barrier(0);
  };
  i32x4 acc[kPanels] = {};
  auto do_step = [&](int s, uint4* stage, bool last) __attribute__((always_inline)) {
    i32x4 a[kPanels][4], c[4];
    wait_step();
    const uint4* const in = stage + wave * kSize;
#pragma unroll
    for (int h = 0; h < 4; ++h) {
      const int at = (4 * h + g) ^ r;
#pragma unroll
      for (int i = 0; i < kPanels; ++i) a[i][h] = *reinterpret_cast<const i32x4*>(in + 16 * (16 * i + r) + at);
      c[h] = *reinterpret_cast<const i32x4*>(in + kW * 64 + 16 * (r % kTokens) + at);
    }
    if (last && KB * (s + 1) > K) {
#pragma unroll
      for (int h = 0; h < 4; ++h) {
        const int left = K - KB * s - 16 * (4 * h + g);        // of these 16 codes, those that count
#pragma unroll
        for (int e = 0; e < 4; ++e)
          c[h][e] &= left >= 4 * e + 4 ? -1 : left <= 4 * e ? 0 : (1 << (8 * (left - 4 * e))) - 1;
      }
    }
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_sched_barrier(0);
    copy_step(s + S, stage);
#pragma unroll
    for (int h = 0; h < 4; ++h)
#pragma unroll
      for (int i = 0; i < kPanels; ++i)
        acc[i] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i][h], c[h], acc[i], 0, 0, 0);
  };
  copy_step(s0, stage0);
  copy_step(s0 + 1, stage1);
  int s = s0;
  for (const int whole = min(s1, K / KB); s + S <= whole; s += S) {
    do_step(s, stage0, false);
    do_step(s + 1, stage1, false);
  }
  if (s < s1) do_step(s, stage0, true);
  if (s + 1 < s1) do_step(s + 1, stage1, true);

  // No copy may still be writing LDS when others write their sums there.
  __builtin_amdgcn_s_waitcnt(0);
  __syncthreads();
  i32x4* const meet = reinterpret_cast<i32x4*>(stage0);
#pragma unroll
  for (int i = 0; i < kPanels; ++i) meet[(4 * i + wave) * 64 + lane] = acc[i];
  __syncthreads();
  // Wavefront i adds up and stores panel i: lane (g, r) holds weight rows
  // 4 g .. 4 g + 3 for token r.
  const int64_t n = n0 + 16 * wave + 4 * g;
  if (wave >= kPanels || n >= p.N || r >= tokens) return;
  float rs[4], bias[4];
  load_int8_rows(p, n, rs, bias);
  const float sb = p.scale[r];
  i32x4 sum = meet[4 * wave * 64 + lane];
#pragma unroll
  for (int k = 1; k < 4; ++k) sum += meet[(4 * wave + k) * 64 + lane];
  store_int8_sums(p, r, n, sb, rs, bias, sum);
}

template <int kTokens, int kPanels>
void enqueue(const Int8Gemm& p, int tiles, hipStream_t stream) {
  hipLaunchKernelGGL((int8_few_kernel<kTokens, kPanels>), dim3((unsigned)tiles), dim3(256), 0, stream, p);
}

}  // namespace

hipError_t launch_int8_few(const Int8Gemm& p, const Int8Plan& plan, hipStream_t stream) {
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
