// 8-bit product y[b][n] = scale[b] row_scale[n] sum_k q[b][k] w[n][k] + bias[n]
// in tiles through LDS, v_mfma_i32_16x16x64_i8, exact 32-bit sums.
//
// A workgroup of 4 wavefronts takes a tile of 32 PN weight rows x 32 PB
// tokens; wavefront (wn, wb) owns PN panels of 16 rows x PB panels of 16
// tokens. The reduction runs in steps of KB bytes, whole cache lines: 128 for
// the large tiles, 256 for the small ones, whose time is that of the weights'
// stream and grows shorter with the runs that a row is read in (27648 x 5120
// at 64 tokens 39 -> 36 us, now 33; 64-byte steps took 51 us at 8192 x 28672, 16
// tokens, where 128 and 256 take 47 and 46). A step's operands are blocks of
// 1 KB, copied straight from memory to LDS (global_load_lds); S stages of LDS
// hold the step in use and those being copied: as many as leave room for the
// workgroups that share a compute unit.
//
// Row r of a panel keeps its 16-byte chunk c at KB r + 16 (c ^ f(r)), f(r) =
// (r & 7) ^ (r >> 3) for 8 chunks, r for 16: any 16 lanes that read the same
// chunk then touch 64 different banks. (The counters show no conflicts for 16
// chunks, and for 8 some, in 18% of the cycles: lanes of two chunks are read
// together. A form of f without any took the same time.)
// The copy of a block puts lane l's 16 bytes at 16 l, so lanes in turn read
// the chunks of one row in the order that f gives: whole lines.
//
// One barrier per step, before its last 64 bytes: passing it, a wavefront knows
// that the next step's stage is full (each waited for its own copies) and
// that this step's has been read into registers by all, so its space takes
// the copies of step s + S. Operands are read 64 bytes ahead, between the
// products, and the copies are spread among the products: bunched up, they
// filled the load unit's queue while the matrix cores waited (8192 x 28672 at
// 2048 tokens 489 -> 404 us). There, by now 340 to 370 us (2.6 to 2.8 POP/s), of
// which the products alone take 280 to 305 and the copies alone 297: the cores
// are busy for 72% of the cycles, at the 1.9 GHz that the card's power leaves
// (alone they hold 3.4 to 3.6 POP/s on random codes, 5 only on zeros).
//
// Few tiles: the reduction is split over ksplit workgroups, whose sums
// int8_join_kernel adds (whole numbers: any order gives the same sum). Up to
// 16 tokens mostly take int8_few.hip's kernel instead.
#include <type_traits>

#include "lq_int8.h"

namespace lq {
namespace {

// A sum as it is used: read here, so that the compiler does not move all of
// them to vector registers (and spill) ahead of the stores.
__device__ __forceinline__ i32x4 acc_take(const i32x4& acc) {
  int v[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) asm volatile("v_accvgpr_read_b32 %0, %1" : "=v"(v[e]) : "a"(acc[e]));
  return (i32x4){v[0], v[1], v[2], v[3]};
}

// acc += a c, in place. (The builtin leaves the choice of the result's
// registers to the compiler: with two steps in a row it took others, and
// moved and spilled 256 sums.) The compiler awaits an asm's operands as before
// any use of them, but knows no product in it and keeps none of a product's
// distances. What keeps them: acc_settle and acc_ready stand between a product
// and whatever else the compiler may do to its sum (moves between the paths
// that meet behind a loop); a product whose addend and result are the result
// of the one right before it (the 32 x 32 tile has a single sum) needs no wait
// at this shape; and operands come from LDS, or are written two instructions
// earlier. tests/test_mfma_asm.py reads all of it out of the compiled kernels,
// along every path: a shape of more passes or another compiler shows there.
__device__ __forceinline__ void mfma_acc(i32x4& acc, i32x4 a, i32x4 c) {
  asm("v_mfma_i32_16x16x64_i8 %0, %1, %2, %0" : "+a"(acc) : "v"(a), "v"(c));
}
__device__ __forceinline__ void mfma_zero(i32x4& acc) {
  acc = (i32x4){0, 0, 0, 0};
  asm("" : "+a"(acc));
}
// 12 and 32 wait states (a product of 4 passes, this one, takes 8, of 8 passes
// 12). Without them the compiler moved sums of the 128-row tiles 5 wait states
// behind their products.
__device__ __forceinline__ void acc_settle() { asm volatile("s_nop 11" ::: "memory"); }
__device__ __forceinline__ void acc_ready() { asm volatile("s_nop 15\n\ts_nop 15" ::: "memory"); }

template <int PN, int PB, int S, int KB>
__global__ __launch_bounds__(256, (PN * PB > 4 ? 1 : 2)) void int8_tile_kernel(
    Int8Gemm p, int tiles_n, int tiles_b, int group_n, int ksplit, int* partial) {
  static_assert(S >= 2 && S <= 4 && (KB == 128 || KB == 256), "stages");
  constexpr int kChunks = KB / 16;             // 16-byte chunks of a row in a step
  constexpr int kCopies = (PN + PB) * KB / 128;   // per wavefront and step, 1 KB each
  constexpr int kBlocks = 4 * kCopies;
  constexpr int kW = PN * KB / 128;            // of a wavefront's copies, those of weights
  __shared__ uint4 stage0[kBlocks * 64];
  __shared__ uint4 stage1[kBlocks * 64];
  __shared__ uint4 stage2[S > 2 ? kBlocks * 64 : 1];
  __shared__ uint4 stage3[S > 3 ? kBlocks * 64 : 1];
  const int lane = threadIdx.x & 63, wave = wave_id();
  const int g = lane >> 4, r = lane & 15;
  const int wn = wave & 1, wb = wave >> 1;

  // Workgroups are dealt to the 8 XCDs in turn: each XCD takes a run of
  // consecutive tiles, and a run goes through group_n tiles of weight rows
  // by all tiles of tokens, so that the tiles at work on an XCD share rows
  // in its L2.
  const int tiles = tiles_n * tiles_b;
  const int per = (tiles * ksplit + 7) / 8;
  const int u = ((int)blockIdx.x & 7) * per + ((int)blockIdx.x >> 3);
  if (u >= tiles * ksplit) return;
  const int t = u % tiles, part_k = __builtin_amdgcn_readfirstlane(u / tiles);
  const TilePlace place = tile_place(t, tiles_n, tiles_b, group_n);
  // (divisions leave the scalar unit: back to it, for scalar addresses)
  const int64_t n0 = (int64_t)__builtin_amdgcn_readfirstlane(place.n) * (32 * PN);
  const int64_t b0 = (int64_t)__builtin_amdgcn_readfirstlane(place.b) * (32 * PB);

  const int K = (int)p.K, K16 = (K + 15) & ~15;
  const int all = (K + KB - 1) / KB, full = K / KB;
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
  const int8_t* const wbase = p.w + n0 * p.ldw;
  const int8_t* const qbase = p.q + b0 * p.ldq;
  uint32_t off[kCopies];
#pragma unroll
  for (int k = 0; k < kCopies; ++k) {
    const int rr = (64 / kChunks) * (wave + 4 * (k < kW ? k : k - kW)) + row;
    off[k] = k < kW ? (uint32_t)min(rr, rows_n - 1) * (uint32_t)p.ldw
                    : (uint32_t)min(rr, rows_b - 1) * (uint32_t)p.ldq;
  }
  auto lane_at = [&](int s) __attribute__((always_inline)) {
    const uint32_t at = (uint32_t)KB * (uint32_t)min(s, steps - 1) + 16u * (uint32_t)chunk;
    return at < (uint32_t)K16 ? at : 0u;
  };
  auto copy_one = [&](int k, uint32_t at, uint4* dst) __attribute__((always_inline)) {
    __builtin_amdgcn_global_load_lds((const void*)((k < kW ? wbase : qbase) + (off[k] + at)),
                                     (__attribute__((address_space(3))) void*)(dst + (wave + 4 * k) * 64), 16,
                                     0, 0);
  };
  auto copy_step = [&](int s, uint4* dst) __attribute__((always_inline)) {
    const uint32_t at = lane_at(s);
#pragma unroll
    for (int k = 0; k < kCopies; ++k) copy_one(k, at, dst);
  };
  // The step that ends inside its KB bytes, if one of this workgroup's does.
  const int part = full < steps && full < all ? full : -1;
  auto zero_past = [&](uint4* st) __attribute__((always_inline)) {
    const int left = K - KB * full - 16 * chunk;       // of this lane's 16 codes, those that count
    if (left >= 16) return;
    uint32_t m[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      m[i] = left >= 4 * i + 4 ? 0xFFFFFFFFu : left <= 4 * i ? 0u : (1u << (8 * (left - 4 * i))) - 1u;
#pragma unroll
    for (int k = kW; k < kCopies; ++k) {
      uint4& c = st[(wave + 4 * k) * 64 + lane];
      c = make_uint4(c.x & m[0], c.y & m[1], c.z & m[2], c.w & m[3]);
    }
  };
  // Units of 16 bytes: row r's chunk 4 h + g (part h of the step, 64 bytes)
  // lies at kChunks r + ((4 h + g) ^ f(r)).
  const int rd = kChunks * r + (g ^ (KB == 128 ? (r & 7) ^ (r >> 3) : r));
  auto rd_part = [&](int h) __attribute__((always_inline)) { return rd ^ (4 * h); };
  const int rd_a = wn * PN * KB, rd_c = (2 * PN + wb * PB) * KB;
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

  i32x4 acc[PN][PB];
#pragma unroll
  for (int i = 0; i < PN; ++i)
#pragma unroll
    for (int j = 0; j < PB; ++j) mfma_zero(acc[i][j]);

  copy_step(s0, stage0);
  copy_step(s0 + 1, stage1);
  if constexpr (S > 2) copy_step(s0 + 2, stage2);
  if constexpr (S > 3) copy_step(s0 + 3, stage3);
  i32x4 a0[PN], c0[PB], a1[PN], c1[PB];
  __builtin_amdgcn_s_waitcnt(kWaitVm0);
  if (part == s0) zero_past(stage0);
  lds_barrier();
#pragma unroll
  for (int i = 0; i < PN; ++i) a0[i] = *reinterpret_cast<const i32x4*>(stage0 + rd_a + rd + KB * i);
#pragma unroll
  for (int j = 0; j < PB; ++j) c0[j] = *reinterpret_cast<const i32x4*>(stage0 + rd_c + rd + KB * j);

  // A part of a step: PN groups of PB products. Each group also issues its
  // share of the reads of the next part's operands (from `next` at rdn), which
  // the last groups need not, and with kFill its share of the copies of step
  // s + S into the stage of step s. Spread like this, they never queue up
  // before the products.
  auto part_step = [&](auto fillc, uint32_t at, uint4* fill, const uint4* next, int rdn, i32x4 (&a)[PN],
                       i32x4 (&c)[PB], i32x4 (&an)[PN], i32x4 (&cn)[PB]) __attribute__((always_inline)) {
    constexpr bool kFill = decltype(fillc)::value;
    constexpr int kEarly = PN > 2 ? PN - 2 : 1;                 // groups that read: done two early
    constexpr int kReads = (PN + PB + kEarly - 1) / kEarly;     // operands per such group
#pragma unroll
    for (int i = 0; i < PN; ++i) {
#pragma unroll
      for (int x = i * kReads; x < (i + 1) * kReads; ++x) {
        if (x < PB) cn[x] = *reinterpret_cast<const i32x4*>(next + rd_c + rdn + KB * x);
        else if (x < PB + PN) an[x - PB] = *reinterpret_cast<const i32x4*>(next + rd_a + rdn + KB * (x - PB));
      }
#pragma unroll
      for (int j = 0; j < PB; ++j) {
        mfma_acc(acc[i][j], a[i], c[j]);
        if constexpr (kFill) {
          // copies k with k * PN * PB / kCopies products before them
#pragma unroll
          for (int k = 0; k < kCopies; ++k)
            if (k * (PN * PB) / kCopies == i * PB + j) copy_one(k, at, fill);
        }
        if (j % 2 == 1 || j == PB - 1) __builtin_amdgcn_sched_barrier(0);
      }
    }
  };
  // One step of KB bytes in parts of 64. Its first part's operands are in a0,
  // c0. Before the last part reads the next step's stage, that stage is full
  // (every wavefront waits for its own copies), and this step's has been read
  // into registers by all and takes the copies of step s + S.
  auto do_step = [&](auto sc, int s) __attribute__((always_inline)) {
    constexpr int su = decltype(sc)::value;
    constexpr int kParts = KB / 64;
    uint4* const cur = stage_c(std::integral_constant<int, su>{});
    uint4* const next = stage_c(std::integral_constant<int, su + 1>{});
    asm volatile("s_nop 1");                    // (a sum may have been cleared right before)
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int h = 0; h + 2 < kParts; h += 2) {
      __builtin_amdgcn_s_waitcnt(kWaitLds0);
      part_step(std::false_type{}, 0u, cur, cur, rd_part(h + 1), a0, c0, a1, c1);
      __builtin_amdgcn_s_waitcnt(kWaitLds0);
      part_step(std::false_type{}, 0u, cur, cur, rd_part(h + 2), a1, c1, a0, c0);
    }
    __builtin_amdgcn_s_waitcnt(kWaitLds0);
    part_step(std::false_type{}, 0u, cur, cur, rd_part(kParts - 1), a0, c0, a1, c1);
    __builtin_amdgcn_s_waitcnt(kWaitVm);
    if (s + 1 == part) zero_past(next);
    lds_barrier();
    part_step(std::true_type{}, lane_at(s + S), cur, next, rd, a1, c1, a0, c0);
  };
  // S steps at a time and one way out of the loop. (The compiler waits for
  // copies of its own accord before it reads where they went, and then for all
  // of them, unless the waits here have told it that they are in. With a test
  // behind each step it lost count and drained them in every round: 512 tokens
  // 8192 x 8192 50 us, not 44.)
  int s = s0;
  for (; s + S <= steps; s += S) {
    do_step(std::integral_constant<int, 0>{}, s);
    do_step(std::integral_constant<int, 1>{}, s + 1);
    if constexpr (S > 2) do_step(std::integral_constant<int, 2>{}, s + 2);
    if constexpr (S > 3) do_step(std::integral_constant<int, 3>{}, s + 3);
    acc_settle();
  }
  auto last_step = [&](auto sc, int s) __attribute__((always_inline)) {
    if (s >= steps) return;
    do_step(sc, s);
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
  if (ksplit > 1) {       // a part of the sums: int8_join_kernel adds the parts
    i32x4* o = reinterpret_cast<i32x4*>(partial) + ((int64_t)u * 4 + wave) * (PN * PB * 64) + lane;
#pragma unroll
    for (int i = 0; i < PN; ++i)
#pragma unroll
      for (int j = 0; j < PB; ++j) o[(i * PB + j) * 64] = acc[i][j];
    return;
  }
  // All scales are loaded before any output is stored. For bf16 two panels of
  // rows are exchanged between lanes of the same token (the upper half of one
  // with the lower half of the other, then odd rows of 16 lanes with even
  // ones) so that lane g holds 8 consecutive outputs of the 32: a token's four
  // lanes store 64 consecutive bytes.
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
        const i32x4 sum = acc_take(acc[i][j]);
        float v[4];
#pragma unroll
        for (int e = 0; e < 4; ++e) v[e] = fmaf((float)sum[e], sb[j] * rs[i][e], bias[i][e]);
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
      if (n < p.N) store_int8_sums(p, b, n, sb[j], rs[i], bias[i], acc_take(acc[i][j]));
    }
  }
}

// The sums of a split reduction: thread (tile, wavefront, panel pair, lane)
// adds the ksplit parts of four outputs and stores them.
template <int PN, int PB>
__global__ __launch_bounds__(256) void int8_join_kernel(Int8Gemm p, int tiles_n, int tiles_b, int group_n,
                                                        int ksplit, const int* partial) {
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
  // (everything is loaded before anything is used: a launch this short is
  // one trip to memory long)
  float rs[4], bias[4];
  load_int8_rows(p, n, rs, bias);
  const float sb = p.scale[b];
  const int64_t stride = (int64_t)tiles * (4 * PN * PB * 64);
  const i32x4* in = reinterpret_cast<const i32x4*>(partial) + id;
  i32x4 v = {0, 0, 0, 0};
  for (int k0 = 0; k0 < ksplit; k0 += 8) {
    i32x4 x[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) x[k] = in[min(k0 + k, ksplit - 1) * stride];
#pragma unroll
    for (int k = 0; k < 8; ++k)
      if (k0 + k < ksplit) v += x[k];
  }
  store_int8_sums(p, b, n, sb, rs, bias, v);
}

}  // namespace

template <int PN, int PB, int S, int KB>
static void enqueue_tile(const Int8Gemm& p, const Int8Plan& plan, int* partial, hipStream_t stream) {
  const int tn = (int)((p.N + 32 * PN - 1) / (32 * PN)), tb = (int)((p.B + 32 * PB - 1) / (32 * PB));
  const int group_n = 4;
  const int per = (tn * tb * plan.ksplit + 7) / 8;
  hipLaunchKernelGGL((int8_tile_kernel<PN, PB, S, KB>), dim3((unsigned)(8 * per)), dim3(256), 0, stream, p, tn,
                     tb, group_n, plan.ksplit, partial);
  if (plan.ksplit > 1)
    hipLaunchKernelGGL((int8_join_kernel<PN, PB>), dim3((unsigned)(tn * tb * PN * PB)), dim3(256), 0,
                       stream, p, tn, tb, group_n, plan.ksplit, partial);
}

// The tiles (stages and bytes per step at the launches below; with `few` those
// of int8_few.hip, four steps at a time), and what they cost in us, fitted to
// 2500 measurements over 180 sizes (1 to 2048 tokens, 60 to 200000 outputs, 150
// to 28672 inputs; profiles/int8_product_times.txt): a step takes `step` plus `share` for every workgroup on
// the compute unit, a workgroup's begin and end take `ends`, and the weights'
// stream, at the rate that its kernel reaches, hides all but kHidden of that
// (or is hidden by it). Of these sizes the choice it gives is on average 0.8%
// above the best of these tiles and splits, 12% at most. Left out, with what
// their absence costs on average: 32 x 64 tokens (0%), a 2-stage 32 x 32 (0.1%).
struct TileCost {
  int rows, tokens, bytes, per_cu;
  float step, share, ends;
  bool few;
};
static constexpr TileCost kTiles[] = {
    {256, 256, 128, 1, 1.155f, 0.167f, 3.9f, false}, {224, 256, 128, 1, 0.932f, 0.262f, 3.1f, false},
    {192, 256, 128, 1, 0.774f, 0.372f, 2.9f, false}, {128, 256, 128, 1, 0.925f, 0.033f, 2.8f, false},
    {128, 128, 128, 1, 0.469f, 0.058f, 2.6f, false}, {128, 64, 256, 1, 0.829f, 0.013f, 2.2f, false},
    {64, 128, 256, 1, 0.530f, 0.323f, 2.1f, false},  {64, 64, 256, 2, 0.728f, 0.225f, 1.5f, false},
    {64, 32, 256, 3, 0.424f, 0.190f, 1.74f, false},  {32, 32, 256, 2, 0.140f, 0.202f, 1.36f, false},
    {16, 4, 1024, 4, 0.369f, 0.511f, 0.72f, true},   {16, 8, 1024, 3, 0.072f, 0.672f, 0.81f, true},
    {16, 16, 1024, 2, 0.112f, 0.593f, 1.12f, true},  {32, 16, 1024, 1, 0.007f, 1.171f, 1.45f, true},
};
constexpr float kJoinUs = 5.0f, kJoinBytesPerUs = 7.0e6f;
constexpr float kStreamBytesPerUs[2] = {4.72e6f, 6.3e6f}, kHidden[2] = {0.216f, 0.298f};     // tiles, few
constexpr int kMaxSplit = 16;
constexpr int64_t kMaxTiles = 1 << 22;    // (a launch has fewer than 2^32 threads)

Int8Plan plan_int8(int64_t B, int64_t N, int64_t K, int cus) {
  if (cus <= 0) cus = 256;
  Int8Plan best{};
  float best_us = 0.0f;
  for (const TileCost& c : kTiles) {
    if (c.few && (B > c.tokens || (c.tokens > 4 && B <= c.tokens / 2))) continue;   // (no more codes than needed)
    const int64_t tiles = ((N + c.rows - 1) / c.rows) * ((B + c.tokens - 1) / c.tokens);
    const float stream = (float)N * (float)K / kStreamBytesPerUs[c.few];      // the weights'
    const int64_t slots = (int64_t)cus * c.per_cu, steps = (K + c.bytes - 1) / c.bytes;
    if (tiles > kMaxTiles && &c != kTiles) continue;
    for (int ks = 1; ks <= kMaxSplit && ks <= steps; ++ks) {
      if (ks > 1 && (c.few || tiles * ks > 4 * (int64_t)cus)) break;
      const float len = (float)((steps + ks - 1) / ks);
      const int64_t units = tiles * ks, full = units / slots, rem = units % slots;
      float us = (float)full * (len * (c.step + c.share * c.per_cu) + c.ends);
      if (rem > 0) {
        const float load = 0.5f * ((float)rem / cus + (float)((rem + cus - 1) / cus));
        us += len * (c.step + c.share * load) + c.ends;
      }
      us = us > stream ? us + kHidden[c.few] * stream : stream + kHidden[c.few] * us;
      const size_t partial = ks > 1 ? (size_t)units * c.rows * c.tokens * 4 : 0;
      if (ks > 1) us += kJoinUs + 2.0f * (float)partial / kJoinBytesPerUs;
      if (best.rows == 0 || us < best_us) {
        best = {c.rows, c.tokens, ks, (int)tiles, c.few, partial};
        best_us = us;
      }
    }
  }
  return best;
}

hipError_t launch_int8_gemm(const Int8Gemm& p, const Int8Plan& plan, int* partial, hipStream_t stream) {
  (void)hipGetLastError();   // clear a stale error of an earlier runtime call
  if (plan.few) return launch_int8_few(p, plan, stream);
  switch (plan.rows / 32 * 16 + plan.tokens / 32) {
    case 0x88: enqueue_tile<8, 8, 2, 128>(p, plan, partial, stream); break;
    case 0x78: enqueue_tile<7, 8, 2, 128>(p, plan, partial, stream); break;
    case 0x68: enqueue_tile<6, 8, 2, 128>(p, plan, partial, stream); break;
    case 0x48: enqueue_tile<4, 8, 2, 128>(p, plan, partial, stream); break;
    case 0x44: enqueue_tile<4, 4, 4, 128>(p, plan, partial, stream); break;
    case 0x42: enqueue_tile<4, 2, 3, 256>(p, plan, partial, stream); break;
    case 0x24: enqueue_tile<2, 4, 3, 256>(p, plan, partial, stream); break;
    case 0x22: enqueue_tile<2, 2, 2, 256>(p, plan, partial, stream); break;
    case 0x21: enqueue_tile<2, 1, 2, 256>(p, plan, partial, stream); break;
    case 0x11: enqueue_tile<1, 1, 4, 256>(p, plan, partial, stream); break;
    default: return hipErrorInvalidValue;
  }
  return hipGetLastError();
}

}  // namespace lq
