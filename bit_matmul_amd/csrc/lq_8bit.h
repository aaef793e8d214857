// The 8-bit layers' and the norms' arguments and launches (arguments as in
// include/lq.h).
#pragma once

#include "lq_internal.h"

namespace lq {

struct QuantRows {
  const void* x;
  const void* gate;      // may be null
  const float* c;        // may be null
  int8_t* q;
  float* scale;
  int64_t B, K, ldx, ldg, ldq;
  int act, lhb;
  float norm;            // 1 / sqrt(hb)
  bool x_bf16;           // x and gate
};
struct NormBlock {
  const void* y;         // may be null, as every pointer below
  const void* gate;
  const float* w_post;
  const void* h;
  void* h_out;
  const float* w_pre;
  void* a;
  int8_t* q;
  float* scale;
  int64_t B, K, ldy, ldg, ldh, ldho, lda, ldq;
  float alpha, eps;
  int act;
  bool y_bf16, h_bf16, a_bf16, post, pre, gate_first, one_plus;
};
struct Int8Gemm {
  const int8_t* q;
  const float* scale;
  const int8_t* w;
  const float* row_scale;
  const float* bias;     // may be null
  void* y;
  int64_t B, N, K, ldq, ldw, ldy;
  bool y_bf16;
};
// How a row kernel holds a row of K values: c blocks of 1024 in each wavefront.
constexpr int kRowBlock = 1024;
constexpr int kRowMaxWaves = 16;
constexpr int kRowMaxC = 4;
constexpr int64_t kRowMaxK = (int64_t)kRowBlock * kRowMaxWaves * kRowMaxC;
struct RowShape {
  int c, waves;
};
RowShape row_shape(int64_t K);
hipError_t launch_quant_rows(const QuantRows& p, hipStream_t stream);
hipError_t launch_norm_block(const NormBlock& p, hipStream_t stream);
// How an 8-bit product runs: tiles of weight rows x tokens, the reduction in
// ksplit parts (more than one: joined by a second launch).
struct Int8Plan {
  int rows, tokens, ksplit, tiles;
  bool few;               // int8_few.hip's kernel
  size_t partial_bytes;   // ksplit > 1: the parts' sums
};
Int8Plan plan_int8(int64_t B, int64_t N, int64_t K, int cus);
// partial: Int8Plan::partial_bytes of workspace (unused when ksplit is 1).
hipError_t launch_int8_gemm(const Int8Gemm& p, const Int8Plan& plan, int* partial, hipStream_t stream);
hipError_t launch_int8_few(const Int8Gemm& p, const Int8Plan& plan, hipStream_t stream);
// Rows and product of one token in one launch (t.q, t.scale and p.q, p.scale
// unused): the weight rows of a workgroup, 0 where it takes two launches.
int int8_token_rows(const QuantRows& t, int64_t N, const Int8Plan& plan);
hipError_t launch_int8_token(const QuantRows& t, const Int8Gemm& p, int rows, hipStream_t stream);

}  // namespace lq
