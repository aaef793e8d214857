// The norm and rotation of queries and keys: arguments and launch (as in
// include/lq.h).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace lq {

constexpr int kQkMaxDim = 512;

struct QkHeads {
  const void* x;
  void* out;
  const float* w;        // may be null
  int64_t ld, ld_head, ldo, ldo_head;
  int heads;
};
struct QkNormRope {
  QkHeads part[2];       // queries, keys
  const void* pos;
  const double* freq;
  int64_t B;
  int dim, rot;
  float eps;
  bool bf16, pos64, norm, one_plus, interleaved;
};
hipError_t launch_qk_norm_rope(const QkNormRope& p, hipStream_t stream);

}  // namespace lq
