// The microscaled 4-bit layers' sizes, arguments and launches (arguments as in
// include/lq.h).
#pragma once

#include "lq_8bit.h"

namespace lq {

constexpr int kMxBlock = 32;         // values that share a scale: 16 bytes of codes
constexpr int kMxUnit = 256;         // values of a panel's run of scales, 128 bytes
constexpr int64_t mx4_units(int64_t K) { return (K + kMxUnit - 1) / kMxUnit; }
constexpr int64_t mx4_row_bytes(int64_t K) { return (K + kMxBlock - 1) / kMxBlock * 16; }
constexpr int64_t mx4_scale_bytes(int64_t rows, int64_t K) { return (rows + 15) / 16 * mx4_units(K) * 128; }

struct Mx4Rows {
  const void* x;
  const void* gate;      // may be null
  const float* c;        // may be null
  uint8_t* q;
  uint8_t* scale;
  int64_t B, K, ldx, ldg, ldq;
  int act, lhb;
  float norm;            // 2^-ceil(lhb / 2)
  bool x_bf16;           // x and gate
};
struct Mx4Gemm {
  const uint8_t* q;
  const uint8_t* scale;
  const uint8_t* w;
  const uint8_t* w_scale;
  const float* row_scale;   // may be null
  const float* bias;        // may be null
  void* y;
  int64_t B, N, K, ldq, ldw, ldy;
  bool y_bf16;
};
hipError_t launch_mx4_rows(const Mx4Rows& p, hipStream_t stream);
// How a 4-bit product runs: the number of its kernel in mx4_gemm.hip's table
// (the last ones mx4_few.hip's), the rest as Int8Plan.
struct Mx4Plan {
  int tile, rows, tokens, ksplit, tiles;
  size_t partial_bytes;
};
Mx4Plan plan_mx4(int64_t B, int64_t N, int64_t K, int cus);
hipError_t launch_mx4_gemm(const Mx4Gemm& p, const Mx4Plan& plan, float* partial, hipStream_t stream);
hipError_t launch_mx4_few(const Mx4Gemm& p, const Mx4Plan& plan, hipStream_t stream);
// Rows and product of one token in one launch (t.q, t.scale and p.q, p.scale
// unused), where it fits and is faster than two.
bool mx4_token_fits(int64_t B, int64_t N, int64_t K, int cus, bool transform, bool gate);
hipError_t launch_mx4_token(const Mx4Rows& t, const Mx4Gemm& p, hipStream_t stream);

}  // namespace lq
