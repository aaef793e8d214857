// 8-bit product for many tokens: y[b][n] = scale[b] row_scale[n] sum_k q[b][k]
// w[n][k] + bias[n], tiles through LDS, v_mfma_i32_16x16x64_i8, exact 32-bit
// sums.
//
// A workgroup of 4 wavefronts takes a tile of 32 PN weight rows x 32 PB
// tokens; wavefront (wn, wb) owns PN panels of 16 rows x PB panels of 16
// tokens. The reduction runs in steps of 64 bytes. A step's operands are
// 2 PN + 2 PB blocks of 1 KB, each the 64 bytes of 16 rows and exactly one
// matrix operand; four stages of LDS hold the step in use and the three
// behind it, copied straight from memory (global_load_lds) three steps
// ahead.
//
// In a block, row r's 16-byte chunk g lies at 64 r + 16 (g ^ f(r)),
// f(r) = (r >> 1 & 3) ^ (r >> 3 & 1): any 8 lanes of consecutive rows that
// read the same chunk then touch 32 different banks, any 16 touch 64. The
// copy of a block puts lane l's 16 bytes at 16 l, so lane l reads chunk
// (l & 3) ^ f(l >> 2) of row l >> 2: four lanes read 64 consecutive bytes.
//
// One barrier per step: passing it, a wavefront knows that the next step's
// stage is filled (each waited for its own copies) and that this step's
// stage has been read into registers by all, so its space is refilled. The
// operands of the next step are read between this step's products.
#include <type_traits>

#include "lq_int8.h"

namespace lq {
namespace {

// acc += a c with acc held in accumulation registers: left to itself the
// compiler spreads 256 sums over both register files and spills. The
// operands were waited for before the step's barrier; the readers of acc
// wait for the last products (acc_ready).
__device__ __forceinline__ void mfma_acc(i32x4& acc, i32x4 a, i32x4 c) {
  acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(a, c, acc, 0, 0, 0);
}
__device__ __forceinline__ void mfma_zero(i32x4& acc) {
  acc = (i32x4){0, 0, 0, 0};
  asm("" : "+a"(acc));
}
__device__ __forceinline__ void acc_ready() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int PN, int PB>
__global__ __launch_bounds__(256, 1) void int8_tile_kernel(Int8Gemm p, int tiles_n, int tiles_b,
                                                           int group_n) {
  constexpr int kBlocks = 2 * PN + 2 * PB;
  constexpr int kCopies = (kBlocks + 3) / 4;
  __shared__ uint4 stage0[kBlocks * 64];
  __shared__ uint4 stage1[kBlocks * 64];
  __shared__ uint4 stage2[kBlocks * 64];
  __shared__ uint4 stage3[kBlocks * 64];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int wn = wave & 1, wb = wave >> 1;

  // Workgroups are dealt to the 8 XCDs in turn: each XCD takes a run of
  // consecutive tiles, and a run goes through group_n tiles of weight rows
  // by all tiles of tokens, so that the tiles at work on an XCD share rows
  // in its L2.
  const int tiles = tiles_n * tiles_b;
  const int per = (tiles + 7) / 8;
  const int t = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (t >= tiles) return;
  const int gsize = group_n * tiles_b;
  const int grp = t / gsize, in = t % gsize;
  const int gn = min(group_n, tiles_n - grp * group_n);
  // (divisions leave the scalar unit: back to it, for scalar addresses)
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(grp * group_n + in % gn) * (32 * PN);
  const int64_t b0 = (int64_t)__builtin_amdgcn_readfirstlane(in / gn) * (32 * PB);

  const int K16 = ((int)p.K + 15) & ~15;
  const int steps = (K16 + 63) / 64, full = K16 / 64;

  // Copy k of this wavefront: block wave + 4 k (past the last block: that one
  // again, the same bytes), this lane's row and chunk of it. Chunks past K
  // (in the last step) are read as the row's first one, and the codes that
  // came that way are then zeroed in LDS by the lanes that copied them.
  const int row = lane >> 2;
  const int chunk = (lane & 3) ^ (((row >> 1) & 3) ^ ((row >> 3) & 1));
  const int rows_n = (int)min((int64_t)(32 * PN), p.N - n0);
  const int rows_b = (int)min((int64_t)(32 * PB), p.B - b0);
  const int8_t* base[kCopies];
  uint32_t off[kCopies];
  int to[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    const int blk = min(wave + 4 * k, kBlocks - 1);
    const bool is_w = blk < 2 * PN;
    const int rr = 16 * (is_w ? blk : blk - 2 * PN) + row;
    base[k] = is_w ? p.w + n0 * p.ldw : p.q + b0 * p.ldq;
    off[k] = (uint32_t)min(rr, (is_w ? rows_n : rows_b) - 1) * (uint32_t)(is_w ? p.ldw : p.ldq);
    to[k] = blk * 64;
  }
  auto lane_at = [&](int s) __attribute__((always_inline)) {
    const uint32_t at = 64u * (uint32_t)min(s, steps - 1) + 16u * (uint32_t)chunk;
    return at < (uint32_t)K16 ? at : 0u;
  };
  auto copy_one = [&](int k, uint32_t at, uint4* dst) __attribute__((always_inline)) {
    __builtin_amdgcn_global_load_lds((const void*)(base[k] + (off[k] + at)),
                                     (__attribute__((address_space(3))) void*)(dst + to[k]), 16, 0, 0);
  };
  auto copy_step = [&](int s, uint4* dst) __attribute__((always_inline)) {
    const uint32_t at = lane_at(s);
#pragma unroll
    for (int k = 0; k < kCopies; ++k) copy_one(k, at, dst);
  };
  // The step that ends inside its 64 bytes, if one does.
  const int part = full < steps ? full : -1;
  auto zero_past = [&](uint4* st) __attribute__((always_inline)) {
#pragma unroll
    for (int k = 0; k < kCopies; ++k)
      if (to[k] >= 2 * PN * 64 && 64 * full + 16 * chunk >= K16) st[to[k] + lane] = make_uint4(0, 0, 0, 0);
  };
  const int rd = 4 * r + (g ^ (((r >> 1) & 3) ^ ((r >> 3) & 1)));   // in 16-byte units
  const int rd_a = wn * PN * 64 + rd, rd_c = (2 * PN + wb * PB) * 64 + rd;
  auto stage_c = [&](auto ic) __attribute__((always_inline)) -> uint4* {
    constexpr int i = decltype(ic)::value & 3;
    if constexpr (i == 0) return stage0;
    else if constexpr (i == 1) return stage1;
    else if constexpr (i == 2) return stage2;
    else return stage3;
  };
  constexpr int kWaitVm = (kCopies & 15) | ((kCopies >> 4) << 14) | (7 << 4) | (15 << 8);
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;

  i32x4 acc[PN][PB];
#pragma unroll
  for (int i = 0; i < PN; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j) mfma_zero(acc[i][j]);

  copy_step(0, stage0);
  copy_step(1, stage1);
  copy_step(2, stage2);
  i32x4 a0[PN], c0[PB], a1[PN], c1[PB];
  __builtin_amdgcn_s_waitcnt((2 * kCopies & 15) | ((2 * kCopies >> 4) << 14) | (7 << 4) | (15 << 8));
  if (part == 0) zero_past(stage0);
  __builtin_amdgcn_s_waitcnt(kWaitLds0);
  __builtin_amdgcn_s_barrier();
#pragma unroll
  for (int i = 0; i < PN; ++i) a0[i] = *reinterpret_cast<const i32x4*>(stage0 + rd_a + 64 * i);
#pragma unroll
  for (int j = 0; j < PB; ++j) c0[j] = *reinterpret_cast<const i32x4*>(stage0 + rd_c + 64 * j);

  // One step: PN groups of PB products. Each group also issues its share of
  // the copies of step s + 3 (into the stage of step s - 1, which every
  // wavefront has read by the barrier) and of the reads of step s + 1's
  // operands, which are done by the last groups. Spread like this, the
  // copies never queue up before the products.
  auto do_step = [&](auto sc, int s, i32x4 (&a)[PN], i32x4 (&c)[PB], i32x4 (&an)[PN],
                     i32x4 (&cn)[PB]) __attribute__((always_inline)) {
    constexpr int su = decltype(sc)::value;
    uint4* const fill = stage_c(std::integral_constant<int, su + 3>{});
    const uint4* const next = stage_c(std::integral_constant<int, su + 1>{});
    constexpr int kReads = (PN + PB + PN - 3) / (PN - 2);       // per group, done two groups early
    constexpr int kPer = (kCopies + PN - 1) / PN;
    const uint32_t at = lane_at(s + 3);
    __builtin_amdgcn_s_waitcnt(kWaitVm);
    if (s + 1 == part) zero_past(stage_c(std::integral_constant<int, su + 1>{}));
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_s_barrier();
#pragma unroll
    for (int i = 0; i < PN; ++i) {
#pragma unroll
      for (int x = i * kReads; x < (i + 1) * kReads; ++x) {
        if (x < PB) cn[x] = *reinterpret_cast<const i32x4*>(next + rd_c + 64 * x);
        else if (x < PB + PN) an[x - PB] = *reinterpret_cast<const i32x4*>(next + rd_a + 64 * (x - PB));
      }
#pragma unroll
      for (int k = i * kPer; k < (i + 1) * kPer; ++k)
        if (k < kCopies) copy_one(k, at, fill);
#pragma unroll
      for (int j = 0; j < PB; ++j)
        mfma_acc(acc[i][j], a[i], c[j]);
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  for (int s = 0;;) {
    do_step(std::integral_constant<int, 0>{}, s, a0, c0, a1, c1);
    if (++s == steps) break;
    do_step(std::integral_constant<int, 1>{}, s, a1, c1, a0, c0);
    if (++s == steps) break;
    do_step(std::integral_constant<int, 2>{}, s, a0, c0, a1, c1);
    if (++s == steps) break;
    do_step(std::integral_constant<int, 3>{}, s, a1, c1, a0, c0);
    if (++s == steps) break;
  }

  // No copy may still be writing LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(0);
  acc_ready();
#pragma unroll
  for (int i = 0; i < PN; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j) asm volatile("" : "+a"(acc[i][j]));
  __builtin_amdgcn_sched_barrier(0);
  // Lane (g, r) of tile (i, j) holds weight rows 4 g .. 4 g + 3 of panel i
  // for token r of panel j. All scales are loaded before any output is
  // stored. For bf16 two panels of rows are exchanged between lanes of the
  // same token (the upper half of one with the lower half of the other, then
  // odd rows of 16 lanes with even ones) so that lane g holds 8 consecutive
  // outputs of the 32: a token's four lanes store 64 consecutive bytes.
  const int64_t nw = n0 + 16 * wn * PN, bw = b0 + 16 * wb * PB + r;
  float rs[PN][4], bias[PN][4], sb[PB];
#pragma unroll
  for (int j = 0; j < PB; ++j) sb[j] = p.scale[min(bw + 16 * j, p.B - 1)];
#pragma unroll
  for (int i = 0; i < PN; ++i) load_int8_rows(p, min(nw + 16 * i + 4 * g, p.N - 1), rs[i], bias[i]);
  if (p.y_bf16 && nw + 16 * PN <= p.N) {
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      const int64_t b = bw + 16 * j;
      uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + b * p.ldy + nw;
      uint32_t w[PN][2];
#pragma unroll
      for (int i = 0; i < PN; ++i) {
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf((float)acc[i][j][e], sb[j] * rs[i][e], bias[i][e]);
        w[i][0] = f32_to_bf16_bits(v[0]) | (f32_to_bf16_bits(v[1]) << 16);
        w[i][1] = f32_to_bf16_bits(v[2]) | (f32_to_bf16_bits(v[3]) << 16);
      }
#pragma unroll
      for (int i = 0; i + 1 < PN; i += 2) {
        uint32_t o[4];
#pragma unroll
        for (int d = 0; d < 2; ++d) {
          const auto x = __builtin_amdgcn_permlane32_swap(w[i][d], w[i + 1][d], false, false);
          const auto z = __builtin_amdgcn_permlane16_swap(x[0], x[1], false, false);
          o[d] = z[0];
          o[2 + d] = z[1];
        }
        if (b < p.B) __builtin_memcpy(y + 16 * i + 8 * g, o, 16);
      }
      if (PN % 2 != 0 && b < p.B) __builtin_memcpy(y + 16 * (PN - 1) + 4 * g, w[PN - 1], 8);
    }
    return;
  }
#pragma unroll
  for (int j = 0; j < PB; ++j) {
    const int64_t b = bw + 16 * j;
    if (b >= p.B) continue;
#pragma unroll
    for (int i = 0; i < PN; ++i) {
      const int64_t n = nw + 16 * i + 4 * g;
      if (n < p.N) store_int8_sums(p, b, n, sb[j], rs[i], bias[i], acc[i][j]);
    }
  }
}

}  // namespace

hipError_t launch_int8_tile(const Int8Gemm& p, hipStream_t stream) {
  const bool big = p.B > 128;
  const int tile = big ? 256 : 128;
  const int tn = (int)((p.N + tile - 1) / tile), tb = (int)((p.B + tile - 1) / tile);
  const int per = (tn * tb + 7) / 8;
  const int group_n = 4;
  if (big)
    hipLaunchKernelGGL((int8_tile_kernel<8, 8>), dim3((unsigned)(8 * per)), dim3(256), 0, stream, p, tn, tb, group_n);
  else
    hipLaunchKernelGGL((int8_tile_kernel<4, 4>), dim3((unsigned)(8 * per)), dim3(256), 0, stream, p, tn, tb, group_n);
  return hipGetLastError();
}

}  // namespace lq
