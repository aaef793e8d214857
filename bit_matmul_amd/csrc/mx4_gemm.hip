// 4-bit product y[b][n] = row_scale[n] sum_k q[b][k] w[n][k] + bias[n] of
// microscaled rows (include/lq.h gives the format) in tiles through LDS,
// v_mfma_scale_f32_16x16x128_f8f6f4: 64 bytes of a row, four blocks, to an
// instruction, which multiplies the blocks' scales in.
//
// The tiles are int8_gemm.hip's, byte for byte: a workgroup of 4 wavefronts
// takes 32 PN weight rows x 32 PB tokens, in steps of KB bytes of every row,
// copied straight from memory to LDS through S stages in the same order of
// chunks; one barrier per step; operands read 64 bytes ahead. With each step
// come its scales, 16 bytes a lane and one copy a wavefront: a panel's 128
// bytes for each 256 values, in which lane (g, r) finds the scales of both its
// blocks (64 bytes apart in the row, byte 0 and 1) at 8 r + 2 g.
//
// Few tiles: the reduction is split over ksplit workgroups, whose sums
// mx4_join_kernel adds in their order.
//
// Sums are the instruction's own, fp32, over 128 values and then in order.
//
// 2048 tokens 8192 -> 28672 230 to 239 us (4.0 to 4.2 PFLOP/s), 28672 -> 8192 192 to 202
// (4.8 to 5.0), of which the matrix cores are busy for 57%, LDS (operands read twice over, copies
// written) for about half. Copies without products take 179 us, products and reads
// without copies 127; codes of nothing but zeros, which cost less power, 12% less.
// One wavefront on a SIMD issues all of it in turn: what gave the copies more time
// was slower (stages of 64 bytes, four of them, 201 -> 218; copies issued half a step
// earlier, with a second barrier, 204 -> 232), and so were smaller tiles, which copy
// more for a product (20480 -> 8192 174 us; in 128 x 128, two to a compute unit, 191,
// in four stages 223). Larger ones than 256 x 256 have no registers for their sums.
// 64 tokens 5120 -> 27648 22 us with its 75 MB of weights from memory (3.4 TB/s), 15.4 where
// the last-level cache holds them.
#include <type_traits>

#include "lq_mx4_mma.h"

namespace lq {
namespace {

// acc += a c, in place, in accumulation registers: inline assembly for the
// reasons that int8_gemm.hip gives for its products (the builtin spilled 268
// registers at 8 x 8 panels), with the same fences: acc_settle and acc_ready
// between a product and whatever else the compiler may do to its sum, a product
// right behind another of the same sum needs no wait at this shape (4 passes),
// operands and scales come from LDS. tests/test_mx4_asm.py reads the distances
// out of the compiled kernels. kHalf: which byte of a lane's scales.
template <int kHalf>
__device__ __forceinline__ void mfma_mx4_acc(f32x4& acc, i32x4 a, i32x4 c, int sa, int sc) {
  if constexpr (kHalf == 0)
    asm("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel_hi:[0,0,0] cbsz:4 blgp:4"
        : "+a"(acc) : "v"(a), "v"(c), "v"(sa), "v"(sc));
  else
    asm("v_mfma_scale_f32_16x16x128_f8f6f4 %0, %1, %2, %0, %3, %4 op_sel:[1,1,0] op_sel_hi:[0,0,0] cbsz:4 blgp:4"
        : "+a"(acc) : "v"(a), "v"(c), "v"(sa), "v"(sc));
}
__device__ __forceinline__ void acc_settle() { asm volatile("s_nop 11" ::: "memory"); }
__device__ __forceinline__ void acc_ready() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

// A sum as it is used (read here: int8_gemm.hip).
__device__ __forceinline__ f32x4 acc_take(const f32x4& acc) {
  float v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[e]) : "a"(acc[e]));
  return (f32x4){v[0], v[1], v[2], v[3]};
}

template <int PN, int PB, int S, int KB>
__global__ __launch_bounds__(256, (PN * PB > 16 || (PN + PB) * KB * S > 2304 ? 1 : 2)) void mx4_tile_kernel(
    Mx4Gemm p, int tiles_n, int tiles_b, int group_n, int ksplit, float* partial) {
  static_assert(S >= 2 && S <= 4 && (KB == 128 || KB == 256), "stages");
  constexpr int kChunks = KB / 16;             // 16-byte chunks, blocks, of a row in a step
  constexpr int kU = KB / 128;                 // runs of scales in a step
  static_assert(kU == 2 || S % 2 == 0, "a step's scales lie in the registers of its parity");
  constexpr int kCodes = (PN + PB) * KB / 128; // copies of codes per wavefront and step, 1 KB each
  constexpr int kBlocks = 4 * kCodes;
  constexpr int kW = PN * KB / 128;            // of a wavefront's copies, those of weights
  // Scales: 2 (PN + PB) panels, kPer of them to a copy of kLane bytes a lane.
  constexpr int kPanels = 2 * (PN + PB);
  constexpr int kLane = kPanels * kU * 128 <= 1024 ? 4 : 16;
  constexpr int kPer = 64 * kLane / (128 * kU);
  constexpr int kScaleCopies = (kPanels + kPer - 1) / kPer;
  static_assert(kScaleCopies <= 4, "one copy of scales to a wavefront");
  constexpr int kCopies = kCodes + 1;
  constexpr int kStage = kBlocks * 64 + kScaleCopies * 4 * kLane;     // 16-byte units
  __shared__ uint4 stage0[kStage];
  __shared__ uint4 stage1[kStage];
  __shared__ uint4 stage2[S > 2 ? kStage : 1];
  __shared__ uint4 stage3[S > 3 ? kStage : 1];
  __shared__ __attribute__((aligned(16))) float outs[2][256];         // the rows' scales and biases
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int wn = wave & 1, wb = wave >> 1;

  // (the order of tiles: int8_gemm.hip)
  const int tiles = tiles_n * tiles_b;
  const int per = (tiles * ksplit + 7) / 8;
  const int u = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (u >= tiles * ksplit) return;
  const int t = u % tiles, part_k = __builtin_amdgcn_readfirstlane(u / tiles);
  const TilePlace place = tile_place(t, tiles_n, tiles_b, group_n);
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(place.n) * (32 * PN);
  const int64_t b0 = (int64_t)__builtin_amdgcn_readfirstlane(place.b) * (32 * PB);

  const int K = (int)p.K, blocks = (K + kMxBlock - 1) / kMxBlock, units = (int)mx4_units(p.K);
  const int all = (blocks + kChunks - 1) / kChunks, full = K / (2 * KB);
  // This workgroup's steps: s0 .. steps - 1.
  const int s0 = (int)((int64_t)all * part_k / ksplit), steps = (int)((int64_t)all * (part_k + 1) / ksplit);

  // Copy k of this wavefront: block wave + 4 k, of 64 / kChunks rows; this
  // lane's row and chunk of it. Chunks past K (in the last step) are read as
  // the row's first one, and the codes that came that way are then zeroed in
  // LDS by the lanes that copied them.
  const int row = lane / kChunks;
  const int panel_row = (wave * (64 / kChunks) + row) & 15;
  const int chunk = (lane % kChunks) ^ (KB == 128 ? (panel_row & 7) ^ (panel_row >> 3) : panel_row);
  const int rows_n = (int)min((int64_t)(32 * PN), p.N - n0);
  const int rows_b = (int)min((int64_t)(32 * PB), p.B - b0);
  const uint8_t* const wbase = p.w + n0 * p.ldw;
  const uint8_t* const qbase = p.q + b0 * p.ldq;
  uint32_t off[kCodes];
#pragma unroll
  for (int k = 0; k < kCodes; ++k) {
    const int rr = (64 / kChunks) * (wave + 4 * (k < kW ? k : k - kW)) + row;
    off[k] = k < kW ? (uint32_t)min(rr, rows_n - 1) * (uint32_t)p.ldw
                    : (uint32_t)min(rr, rows_b - 1) * (uint32_t)p.ldq;
  }
  // Scales: this wavefront's copy (the last one, where there are fewer than
  // wavefronts: the same bytes to the same place) and this lane's panel of it,
  // those that do not exist as the last one.
  const int scopy = min(wave, kScaleCopies - 1);
  constexpr int kLanesPer = 64 / kPer;
  const int spanel = scopy * kPer + lane / kLanesPer, sunit = lane % kLanesPer * kLane / 128;
  const uint8_t* sbase;
  {
    const bool is_w = spanel < 2 * PN;
    const int64_t last = ((is_w ? p.N : p.B) - 1) / 16;
    const int64_t panel = min((is_w ? n0 / 16 + spanel : b0 / 16 + (spanel - 2 * PN)), last);
    sbase = (is_w ? p.w_scale : p.scale) + panel * ((int64_t)units * 128) + lane % kLanesPer * kLane % 128;
  }
  auto lane_at = [&](int s) __attribute__((always_inline)) {
    const int blk = kChunks * min(s, steps - 1) + chunk;
    return blk < blocks ? 16u * (uint32_t)blk : 0u;
  };
  auto copy_one = [&](int k, int s, uint32_t at, uint4* dst) __attribute__((always_inline)) {
    if (k < kCodes) {
      __builtin_amdgcn_global_load_lds((const void*)((k < kW ? wbase : qbase) + (off[k] + at)),
                                       (__attribute__((address_space(3))) void*)(dst + (wave + 4 * k) * 64), 16,
                                       0, 0);
    } else {
      const int unit = min(kU * min(s, steps - 1) + sunit, units - 1);
      const auto from = (const void*)(sbase + 128u * (uint32_t)unit);
      const auto to = (__attribute__((address_space(3))) void*)(dst + kBlocks * 64 + scopy * 4 * kLane);
      if constexpr (kLane == 4) __builtin_amdgcn_global_load_lds(from, to, 4, 0, 0);
      else __builtin_amdgcn_global_load_lds(from, to, 16, 0, 0);
    }
  };
  auto copy_step = [&](int s, uint4* dst) __attribute__((always_inline)) {
    const uint32_t at = lane_at(s);
#pragma unroll
    for (int k = 0; k < kCopies; ++k) copy_one(k, s, at, dst);
  };
  // The step that ends inside its KB bytes, if one of this workgroup's does.
  const int part = full < steps && full < all ? full : -1;
  // What lies past K there: codes of tokens as zero, and scales of both sides
  // (a NaN times zero would not vanish).
  auto zero_past = [&](uint4* st) __attribute__((always_inline)) {
    const int left = K - 2 * KB * full - 32 * chunk;       // of this lane's 32 codes, those that count
    if (left < 32) {
#pragma unroll
      for (int k = kW; k < kCodes; ++k) {
        uint4& c = st[(wave + 4 * k) * 64 + lane];
        c = make_uint4(c.x & mx4_mask(left, 0), c.y & mx4_mask(left, 1), c.z & mx4_mask(left, 2), c.w & mx4_mask(left, 3));
      }
    }
    const int sleft = blocks - 8 * (kU * full + sunit);
    uint32_t* const w = reinterpret_cast<uint32_t*>(st + kBlocks * 64 + scopy * 4 * kLane) + lane * (kLane / 4);
#pragma unroll
    for (int i = 0; i < kLane / 4; ++i) w[i] &= mx4_scale_mask(sleft, kLane == 4 ? lane & 1 : i & 1);
  };
  // Units of 16 bytes: row r's chunk 4 h + g (part h of the step, 64 bytes)
  // lies at kChunks r + ((4 h + g) ^ f(r)).
  const int rd = kChunks * r + (g ^ (KB == 128 ? (r & 7) ^ (r >> 3) : r));
  auto rd_part = [&](int h) __attribute__((always_inline)) { return rd ^ (4 * h); };
  const int rd_a = wn * PN * KB, rd_c = (2 * PN + wb * PB) * KB;
  const int rd_s = 4 * r + g;                  // scales, of 2 bytes
  auto stage_c = [&](auto ic) __attribute__((always_inline)) -> uint4* {
    constexpr int i = decltype(ic)::value % S;
    if constexpr (i == 0) return stage0;
    else if constexpr (i == 1) return stage1;
    else if constexpr (i == 2) return stage2;
    else return stage3;
  };
  constexpr int kVm = (S - 2) * kCopies;      // copies behind the next step's at a step's barrier
  constexpr int kVm0 = (S - 1) * kCopies;     // behind the first step's before the loop
  static_assert(kVm0 < 64, "the counter of loads in flight");
  constexpr int kWaitVm = (kVm & 15) | ((kVm >> 4) << 14) | (7 << 4) | (15 << 8);
  constexpr int kWaitVm0 = (kVm0 & 15) | ((kVm0 >> 4) << 14) | (7 << 4) | (15 << 8);
  constexpr int kWaitLds0 = (3 << 14) | (7 << 4) | 15;

  f32x4 acc[PN][PB];
#pragma unroll
  for (int i = 0; i < PN; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      acc[i][j] = (f32x4){0.0f, 0.0f, 0.0f, 0.0f};
      asm("" : "+a"(acc[i][j]));
    }

  // The rows' scales and biases, here: behind the loop they were one trip to
  // memory after another. (Threads past the tile's rows: the last row's.)
  const int64_t out = min(n0 + (int)threadIdx.x, p.N - 1);
  const float out_scale = p.row_scale != nullptr ? p.row_scale[out] : 1.0f;
  const float out_bias = p.bias != nullptr ? p.bias[out] : 0.0f;
  __builtin_amdgcn_sched_barrier(0);
  copy_step(s0, stage0);
  copy_step(s0 + 1, stage1);
  if constexpr (S > 2) copy_step(s0 + 2, stage2);
  if constexpr (S > 3) copy_step(s0 + 3, stage3);
  i32x4 a0[PN], c0[PB], a1[PN], c1[PB];
  int sa[2][PN], sc[2][PB];                   // of runs of scales, in turn
  __builtin_amdgcn_s_waitcnt(kWaitVm0);
  if (part == s0) zero_past(stage0);
  lds_barrier();
  auto scale_a = [&](const uint4* st, int run, int i) __attribute__((always_inline)) -> int {
    return reinterpret_cast<const uint16_t*>(st + kBlocks * 64)[((wn * PN + i) * kU + run) * 64 + rd_s];
  };
  auto scale_c = [&](const uint4* st, int run, int j) __attribute__((always_inline)) -> int {
    return reinterpret_cast<const uint16_t*>(st + kBlocks * 64)[((2 * PN + wb * PB + j) * kU + run) * 64 + rd_s];
  };
#pragma unroll
  for (int i = 0; i < PN; ++i) {
    a0[i] = *reinterpret_cast<const i32x4*>(stage0 + rd_a + rd + KB * i);
    sa[0][i] = scale_a(stage0, 0, i);
  }
#pragma unroll
  for (int j = 0; j < PB; ++j) {
    c0[j] = *reinterpret_cast<const i32x4*>(stage0 + rd_c + rd + KB * j);
    sc[0][j] = scale_c(stage0, 0, j);
  }

  // A part of a step: PN groups of PB products. Each group also issues its
  // share of the reads of the next part's operands (from `next` at rdn, with
  // the scales of its run where it begins one), which the last groups need
  // not, and with kFill its share of the copies of step s + S into the stage
  // of step s.
  auto part_step = [&](auto fillc, auto halfc, int s, uint32_t at, uint4* fill, const uint4* next, int rdn, int run,
                       i32x4 (&a)[PN], i32x4 (&c)[PB], i32x4 (&an)[PN], i32x4 (&cn)[PB], int (&ma)[PN], int (&mc)[PB],
                       int (&man)[PN], int (&mcn)[PB]) __attribute__((always_inline)) {
    constexpr bool kFill = decltype(fillc)::value;
    constexpr int kHalf = decltype(halfc)::value;               // which of a lane's two scales
    constexpr int kEarly = PN > 2 ? PN - 2 : 1;                 // groups that read: done two early
    constexpr int kReads = (PN + PB + kEarly - 1) / kEarly;     // operands per such group
#pragma unroll
    for (int i = 0; i < PN; ++i) {
#pragma unroll
      for (int x = i * kReads; x < (i + 1) * kReads; ++x) {
        if (x < PB) {
          cn[x] = *reinterpret_cast<const i32x4*>(next + rd_c + rdn + KB * x);
          if constexpr (kHalf == 1) mcn[x] = scale_c(next, run, x);
        } else if (x < PB + PN) {
          an[x - PB] = *reinterpret_cast<const i32x4*>(next + rd_a + rdn + KB * (x - PB));
          if constexpr (kHalf == 1) man[x - PB] = scale_a(next, run, x - PB);
        }
      }
#pragma unroll
      for (int j = 0; j < PB; ++j) {
        mfma_mx4_acc<kHalf>(acc[i][j], a[i], c[j], ma[i], mc[j]);
        if constexpr (kFill) {
          // copies k with k * PN * PB / kCopies products before them
#pragma unroll
          for (int k = 0; k < kCopies; ++k)
            if (k * (PN * PB) / kCopies == i * PB + j) copy_one(k, s + S, at, fill);
        }
        if (j % 2 == 1 || j == PB - 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // One step of KB bytes in parts of 64. Its first part's operands are in a0,
  // c0, its first scales in sa[su % 2], sc[su % 2] (KB 128) or sa[0], sc[0].
  // The order of waits, barrier and copies is int8_gemm.hip's.
  auto do_step = [&](auto sc_, int s) __attribute__((always_inline)) {
    constexpr int su = decltype(sc_)::value;
    uint4* const cur = stage_c(std::integral_constant<int, su>{});
    uint4* const next = stage_c(std::integral_constant<int, su + 1>{});
    using H0 = std::integral_constant<int, 0>;
    using H1 = std::integral_constant<int, 1>;
    asm volatile("s_nop 1");                    // (a sum may have been cleared right before)
    __builtin_amdgcn_sched_barrier(0);
    if constexpr (kU == 2) {
      __builtin_amdgcn_s_waitcnt(kWaitLds0);
      part_step(std::false_type{}, H0{}, s, 0u, cur, cur, rd_part(1), 0, a0, c0, a1, c1, sa[0], sc[0], sa[1], sc[1]);
      __builtin_amdgcn_s_waitcnt(kWaitLds0);
      part_step(std::false_type{}, H1{}, s, 0u, cur, cur, rd_part(2), 1, a1, c1, a0, c0, sa[0], sc[0], sa[1], sc[1]);
    }
    constexpr int m = kU == 2 ? 1 : su % 2;
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    part_step(std::false_type{}, H0{}, s, 0u, cur, cur, rd_part(2 * kU - 1), 0, a0, c0, a1, c1, sa[m], sc[m], sa[1 - m],
              sc[1 - m]);
    __builtin_amdgcn_s_waitcnt(kWaitVm);
    if (s + 1 == part) zero_past(next);
    lds_barrier();
    part_step(std::true_type{}, H1{}, s, lane_at(s + S), cur, next, rd, 0, a1, c1, a0, c0, sa[m], sc[m], sa[1 - m],
              sc[1 - m]);
  };
  // S steps at a time and one way out of the loop (int8_gemm.hip).
  int s = s0;
  for (; s + S <= steps; s += S) {
    do_step(std::integral_constant<int, 0>{}, s);
    do_step(std::integral_constant<int, 1>{}, s + 1);
    if constexpr (S > 2) do_step(std::integral_constant<int, 2>{}, s + 2);
    if constexpr (S > 3) do_step(std::integral_constant<int, 3>{}, s + 3);
    acc_settle();
  }
  auto last_step = [&](auto sc_, int s) __attribute__((always_inline)) {
    if (s >= steps) return;
    do_step(sc_, s);
    acc_settle();
  };
  last_step(std::integral_constant<int, 0>{}, s);
  if constexpr (S > 2) last_step(std::integral_constant<int, 1>{}, s + 1);
  if constexpr (S > 3) last_step(std::integral_constant<int, 2>{}, s + 2);

  // No copy may still be writing LDS when the workgroup ends.
  __builtin_amdgcn_s_waitcnt(0);
  acc_ready();
#pragma unroll
  for (int i = 0; i < PN; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j) asm volatile("" : "+a"(acc[i][j]));
  __builtin_amdgcn_sched_barrier(0);
  // Lane (g, r) of tile (i, j) holds weight rows 4 g .. 4 g + 3 of panel i
  // for token r of panel j.
  if (ksplit > 1) {       // a part of the sums: mx4_join_kernel adds the parts
    f32x4* o = reinterpret_cast<f32x4*>(partial) + ((int64_t)u * 4 + wave) * (PN * PB * 64) + lane;
#pragma unroll
    for (int i = 0; i < PN; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j) o[(i * PB + j) * 64] = acc[i][j];
    return;
  }
  outs[0][threadIdx.x] = out_scale;
  outs[1][threadIdx.x] = out_bias;
  lds_barrier();
  // (pairs of panels exchanged so that a token's four lanes store
  // 64 consecutive bytes: int8_gemm.hip)
  const int64_t nw = n0 + 16 * wn * PN, bw = b0 + 16 * wb * PB + r;
  float rs[PN][4], bias[PN][4];
#pragma unroll
  for (int i = 0; i < PN; ++i) {
    __builtin_memcpy(rs[i], &outs[0][16 * (wn * PN + i) + 4 * g], 16);
    __builtin_memcpy(bias[i], &outs[1][16 * (wn * PN + i) + 4 * g], 16);
  }
  if (p.y_bf16 && nw + 16 * PN <= p.N) {
#pragma unroll
    for (int j = 0; j < PB; ++j) {
      const int64_t b = bw + 16 * j;
      uint16_t* y = reinterpret_cast<uint16_t*>(p.y) + b * p.ldy + nw;
      uint32_t w[PN][2];
#pragma unroll
      for (int i = 0; i < PN; ++i) {
        const f32x4 sum = acc_take(acc[i][j]);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf(sum[e], rs[i][e], bias[i][e]);
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
      __builtin_amdgcn_sched_barrier(0);      // (one panel of tokens in registers at a time)
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
      if (n < p.N) store_mx4_sums(p, b, n, rs[i], bias[i], acc_take(acc[i][j]));
    }
  }
}

// The sums of a split reduction: thread (tile, wavefront, panel pair, lane)
// adds the ksplit parts of four outputs, in their order, and stores them.
template <int PN, int PB>
__global__ __launch_bounds__(256) void mx4_join_kernel(Mx4Gemm p, int tiles_n, int tiles_b, int group_n,
                                                       int ksplit, const float* partial) {
  const int tiles = tiles_n * tiles_b;
  const int64_t id = (int64_t)blockIdx.x * 256 + threadIdx.x;
  const int lane = threadIdx.x & 63;
  const int64_t rest = id >> 6;
  const int ij = (int)(rest % (PN * PB)), wave = (int)(rest / (PN * PB)) & 3;
  const int t = (int)(rest / (4 * PN * PB));
  if (t >= tiles) return;
  const TilePlace at = tile_place(t, tiles_n, tiles_b, group_n);
  const int64_t n = (int64_t)at.n * (32 * PN) + 16 * ((wave & 1) * PN + ij / PB) + 4 * (lane >> 4);
  const int64_t b = (int64_t)at.b * (32 * PB) + 16 * ((wave >> 1) * PB + ij % PB) + (lane & 15);
  if (n >= p.N || b >= p.B) return;
  float rs[4], bias[4];
  load_mx4_rows(p, n, rs, bias);
  const int64_t stride = (int64_t)tiles * (4 * PN * PB * 64);
  const f32x4* in = reinterpret_cast<const f32x4*>(partial) + id;
  f32x4 v = {0.0f, 0.0f, 0.0f, 0.0f};
  for (int k0 = 0; k0 < ksplit; k0 += 8) {
    f32x4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = in[min(k0 + k, ksplit - 1) * stride];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k0 + k < ksplit) v += x[k];
  }
  store_mx4_sums(p, b, n, rs, bias, v);
}

template <int PN, int PB, int S, int KB>
void enqueue_tile(const Mx4Gemm& p, const Mx4Plan& plan, float* partial, hipStream_t stream) {
  const int tn = (int)((p.N + 32 * PN - 1) / (32 * PN)), tb = (int)((p.B + 32 * PB - 1) / (32 * PB));
  const int group_n = 4;
  const int per = (tn * tb * plan.ksplit + 7) / 8;
  hipLaunchKernelGGL((mx4_tile_kernel<PN, PB, S, KB>), dim3((unsigned)(8 * per)), dim3(256), 0, stream, p, tn,
                     tb, group_n, plan.ksplit, partial);
  if (plan.ksplit > 1)
    hipLaunchKernelGGL((mx4_join_kernel<PN, PB>), dim3((unsigned)(tn * tb * PN * PB)), dim3(256), 0,
                       stream, p, tn, tb, group_n, plan.ksplit, partial);
}

// The tiles, by their number (launch_mx4_gemm), and what they cost in us, fitted
// to 25000 measurements over 1278 sizes (1 to 2048 tokens, 16 to 65536 outputs,
// 64 to 28672 inputs; some of them in profiles/mx4_product_times.txt): a step
// takes `step` plus `share` for every workgroup on the compute unit, a
// workgroup's begin and end take `ends`, and the weights' stream comes on top at
// its kernel's rate; rows that are no whole cache lines long take kRagged more. With the
// time of its own choice measured at every size, that is 1.2% above the best of these tiles
// and splits on average and 17% at most at 317 of those sizes, 1.6% and 17% at 150 others.
// Left out, with what their absence costs on average: 128 x 256 tokens (0%),
// 64 x 128 (0.1%), 128 x 64 in 3 steps of 256 bytes (0.1%), 64 x 64 in 2 (0%).
struct TileCost {
  int rows, tokens, bytes, per_cu;
  float step, share, ends;
  bool few;
};
constexpr TileCost kTiles[] = {
    {256, 256, 128, 1, 0.257f, 1.406f, 8.80f, false}, {224, 256, 128, 1, 0.381f, 1.138f, 8.79f, false},
    {192, 256, 128, 1, 0.404f, 0.933f, 8.91f, false}, {128, 128, 128, 1, 0.307f, 0.215f, 5.31f, false},
    {128, 128, 128, 2, 0.300f, 0.406f, 4.18f, false}, {128, 64, 128, 1, 0.299f, 0.034f, 3.89f, false},
    {64, 64, 128, 2, 0.080f, 0.160f, 3.71f, false}, {64, 32, 256, 1, 0.291f, 0.000f, 3.81f, false},
    {64, 32, 128, 2, 0.118f, 0.128f, 3.58f, false}, {32, 32, 256, 2, 0.107f, 0.126f, 3.74f, false},
    {16, 4, 1024, 4, 0.058f, 0.437f, 2.90f, true}, {16, 8, 1024, 3, 0.145f, 0.265f, 2.36f, true},
    {16, 16, 1024, 2, 0.214f, 0.312f, 2.88f, true}, {32, 16, 1024, 1, 0.486f, 0.268f, 2.89f, true},
};
constexpr float kJoinUs = 2.31f, kJoinBytesPerUs = 5.83e+06f, kRagged = 0.144f;
constexpr float kStreamBytesPerUs[2] = {7.579e+06f, 9.369e+06f};     // tiles, few
constexpr int kMaxSplit = 16;
constexpr int64_t kMaxTiles = 1 << 22;    // (a launch has fewer than 2^32 threads)

}  // namespace

// (A call makes its plan: 32-bit arithmetic, and of a tile no more splits than
// could fill the device. At most 2^26 workgroups and 2^13 steps.)
Mx4Plan plan_mx4(int64_t B, int64_t N, int64_t K, int cus) {
  if (cus <= 0) cus = 256;
  Mx4Plan best{};
  float best_us = 0.0f;
  const uint32_t bytes = (uint32_t)mx4_row_bytes(K), ucus = (uint32_t)cus;
  const float ragged = bytes % 128 != 0 ? 1.0f + kRagged : 1.0f;
  for (const TileCost& c : kTiles) {
    if (c.few && (B > c.tokens || (c.tokens > 4 && B <= c.tokens / 2))) continue;   // (no more codes than needed)
    // (Wide tiles of mostly no tokens lie outside of what the costs were fitted to, which put them too
    // low: 24 tokens 512 -> 65536 9.6 us, in 32-token tiles 9.4; 8 tokens 1024 -> 65536 13.5 and 12.5; one
    // token 11008 -> 65536 in 64-token tiles 70.7, in 32-token ones 67.2.)
    if (c.tokens >= 128 ? c.tokens >= 4 * B : c.tokens >= 64 * B) continue;
    const uint32_t tiles_n = ((uint32_t)N + c.rows - 1) / c.rows, tiles_b = ((uint32_t)B + c.tokens - 1) / c.tokens;
    if ((uint64_t)tiles_n * tiles_b > (uint64_t)kMaxTiles && &c != kTiles) continue;
    const uint32_t tiles = tiles_n * tiles_b, slots = ucus * c.per_cu, steps = (bytes + c.bytes - 1) / c.bytes;
    const float stream = (float)N * (float)bytes / kStreamBytesPerUs[c.few];      // the weights'
    uint32_t most = c.few ? 1u : 4u * ucus / tiles;
    most = most < 1u ? 1u : most > (uint32_t)kMaxSplit ? (uint32_t)kMaxSplit : most;
    for (uint32_t ks = 1; ks <= most && ks <= steps; ++ks) {
      const float len = ragged * (float)((steps + ks - 1) / ks);
      const uint32_t units = tiles * ks, full = units / slots, rem = units - full * slots;
      float us = ragged * stream + (float)full * (len * (c.step + c.share * c.per_cu) + c.ends);
      if (rem > 0) {
        const float load = 0.5f * ((float)rem / (float)ucus + (float)((rem + ucus - 1) / ucus));
        us += len * (c.step + c.share * load) + c.ends;
      }
      const size_t partial = ks > 1 ? (size_t)units * c.rows * c.tokens * 4 : 0;
      if (ks > 1) us += kJoinUs + 2.0f * (float)partial / kJoinBytesPerUs;
      if (best.rows == 0 || us < best_us) {
        best = {(int)(&c - kTiles), c.rows, c.tokens, (int)ks, (int)tiles, partial};
        best_us = us;
      }
    }
  }
  return best;
}

hipError_t launch_mx4_gemm(const Mx4Gemm& p, const Mx4Plan& plan, float* partial, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  switch (plan.tile) {
    case 0: enqueue_tile<8, 8, 2, 128>(p, plan, partial, stream); break;
    case 1: enqueue_tile<7, 8, 2, 128>(p, plan, partial, stream); break;
    case 2: enqueue_tile<6, 8, 2, 128>(p, plan, partial, stream); break;
    case 3: enqueue_tile<4, 4, 4, 128>(p, plan, partial, stream); break;
    case 4: enqueue_tile<4, 4, 2, 128>(p, plan, partial, stream); break;
    case 5: enqueue_tile<4, 2, 4, 128>(p, plan, partial, stream); break;
    case 6: enqueue_tile<2, 2, 4, 128>(p, plan, partial, stream); break;
    case 7: enqueue_tile<2, 1, 4, 256>(p, plan, partial, stream); break;
    case 8: enqueue_tile<2, 1, 4, 128>(p, plan, partial, stream); break;
    case 9: enqueue_tile<1, 1, 4, 256>(p, plan, partial, stream); break;
    default: return launch_mx4_few(p, plan, stream);
  }
  return hipGetLastError();
}

}  // namespace lq
