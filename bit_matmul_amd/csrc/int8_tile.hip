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

// 16 zero bytes for the chunks of q past K.
__device__ const uint4 kZeroChunk = {0, 0, 0, 0};

template <int PN, int PB>
__global__ __launch_bounds__(256, 1) void int8_tile_kernel(Int8Gemm p, int tiles_n, int tiles_b,
                                                           int group_n) {
  constexpr int kBlocks = 2 * PN + 2 * PB;
  constexpr int kCopies = kBlocks / 4;
  constexpr int kStages = 4;
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
  if (((int)blockIdx.x >> 3) >= per || t >= tiles) return;
  const int gsize = group_n * tiles_b;
  const int grp = t / gsize, in = t % gsize;
  const int gn = min(group_n, tiles_n - grp * group_n);
  const int64_t n0 = (int64_t)(grp * group_n + in % gn) * (32 * PN);
  const int64_t b0 = (int64_t)(in / gn) * (32 * PB);

  const int K16 = ((int)p.K + 15) & ~15;
  const int steps = (K16 + 63) / 64;

  // Copy k of this wavefront: block wave + 4 k; its lane's row and chunk.
  const int row = lane >> 2;
  const int chunk = (lane & 3) ^ (((row >> 1) & 3) ^ ((row >> 3) & 1));
  const int8_t* const wbase = p.w + n0 * p.ldw;
  const int8_t* const qbase = p.q + b0 * p.ldq;
  const int rows_n = (int)min((int64_t)(32 * PN), p.N - n0);
  const int rows_b = (int)min((int64_t)(32 * PB), p.B - b0);
  uint32_t off[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    const int blk = wave + 4 * k;
    const bool is_w = k < PN / 2;
    const int rr = 16 * (is_w ? blk : blk - 2 * PN) + row;
    off[k] = is_w ? (uint32_t)min(rr, rows_n - 1) * (uint32_t)p.ldw + 16 * chunk
                  : (uint32_t)min(rr, rows_b - 1) * (uint32_t)p.ldq + 16 * chunk;
  }
  auto copy_step = [&](int s, uint4* dst) __attribute__((always_inline)) {
    const int at = 64 * min(s, steps - 1);
    auto copy = [&](const int8_t* from, int k) __attribute__((always_inline)) {
      __builtin_amdgcn_global_load_lds((const void*)from,
                                       (__attribute__((address_space(3))) void*)(dst + (wave + 4 * k) * 64),
                                       16, 0, 0);
    };
    if (at + 64 <= K16) {
#pragma unroll
      for (int k = 0; k < kCopies; ++k) {
        const int8_t* src = (k < PN / 2 ? wbase : qbase) + at;
        copy(src + off[k], k);
      }
    } else {
      // chunks past K: zero codes, against any weights that are there
      const bool past = at + 16 * chunk >= K16;
#pragma unroll
      for (int k = 0; k < kCopies; ++k) {
        const bool is_w = k < PN / 2;
        const int8_t* from = (is_w ? wbase : qbase) + off[k] + (past ? -16 * chunk : at);
        if (!is_w && past) from = reinterpret_cast<const int8_t*>(&kZeroChunk);
        copy(from, k);
      }
    }
  };
  const int rd = 4 * r + (g ^ (((r >> 1) & 3) ^ ((r >> 3) & 1)));   // in 16-byte units
  auto read_step = [&](const uint4* st, i32x4 (&a)[PN], i32x4 (&c)[PB]) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < PN; ++i) a[i] = *reinterpret_cast<const i32x4*>(st + (wn * PN + i) * 64 + rd);
#pragma unroll
    for (int j = 0; j < PB; ++j)
      c[j] = *reinterpret_cast<const i32x4*>(st + (2 * PN + wb * PB + j) * 64 + rd);
  };
  auto stage_c = [&](auto ic) __attribute__((always_inline)) -> uint4* {
    constexpr int i = decltype(ic)::value & 3;
    if constexpr (i == 0) return stage0;
    else if constexpr (i == 1) return stage1;
    else if constexpr (i == 2) return stage2;
    else return stage3;
  };
  constexpr int kVm = (kStages - 2) * kCopies;        // copies that may be in flight at the barrier
  constexpr int kWaitVm = (kVm & 15) | ((kVm >> 4) << 14) | (7 << 4) | (15 << 8);
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;

  i32x4 acc[PN][PB];
#pragma unroll
  for (int i = 0; i < PN; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j) acc[i][j] = (i32x4){0, 0, 0, 0};

  copy_step(0, stage0);
  copy_step(1, stage1);
  copy_step(2, stage2);
  i32x4 a0[PN], c0[PB], a1[PN], c1[PB];
  __builtin_amdgcn_s_waitcnt(kWaitVm);
  __builtin_amdgcn_s_barrier();
  read_step(stage0, a0, c0);

  auto do_step = [&](auto sc, int s, i32x4 (&a)[PN], i32x4 (&c)[PB], i32x4 (&an)[PN],
                     i32x4 (&cn)[PB]) __attribute__((always_inline)) {
    constexpr int su = decltype(sc)::value;
    // The next step's stage (copied two steps ago or earlier), and this
    // wavefront's reads of this step's.
    copy_step(s + 3, stage_c(std::integral_constant<int, su + 3>{}));
    __builtin_amdgcn_s_waitcnt(kWaitVm);
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    __builtin_amdgcn_s_barrier();
    read_step(stage_c(std::integral_constant<int, su + 1>{}), an, cn);
#pragma unroll
    for (int i = 0; i < PN; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j)
        acc[i][j] = __builtin_amdgcn_mfma_i32_16x16x64_i8(a[i], c[j], acc[i][j], 0, 0, 0);
  };
  int s = 0;
  for (; s + 4 <= steps; s += 4) {
    do_step(std::integral_constant<int, 0>{}, s, a0, c0, a1, c1);
    do_step(std::integral_constant<int, 1>{}, s + 1, a1, c1, a0, c0);
    do_step(std::integral_constant<int, 2>{}, s + 2, a0, c0, a1, c1);
    do_step(std::integral_constant<int, 3>{}, s + 3, a1, c1, a0, c0);
  }
  if (s < steps) do_step(std::integral_constant<int, 0>{}, s, a0, c0, a1, c1);
  if (s + 1 < steps) do_step(std::integral_constant<int, 1>{}, s + 1, a1, c1, a0, c0);
  if (s + 2 < steps) do_step(std::integral_constant<int, 2>{}, s + 2, a0, c0, a1, c1);

  // No copy may still be writing LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(0);
  // Lane (g, r) of tile (i, j) holds weight rows 4 g .. 4 g + 3 of panel i
  // for token r of panel j.
#pragma unroll
  for (int j = 0; j < PB; ++j) {
    const int64_t b = b0 + 16 * (wb * PB + j) + r;
    if (b >= p.B) continue;
    const float sb = p.scale[b];
#pragma unroll
    for (int i = 0; i < PN; ++i) {
      const int64_t n = n0 + 16 * (wn * PN + i) + 4 * g;
      if (n >= p.N) continue;
      store_int8_sums(p, b, n, sb, acc[i][j]);
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
