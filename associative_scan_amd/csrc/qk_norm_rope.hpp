// Private interface between the C ABI and the query / key norm kernels.
#pragma once

#include "la_launch.hpp"

namespace mscan {
namespace la {

struct NormProblem {
  int64_t B, T;
  int32_t D, rot;          // head size, rotated entries (a multiple of 16)
  int32_t interleaved;     // pairs (2i, 2i + 1) instead of (i, i + rot / 2)
  float eps;
  const float *cos, *sin;  // [table][rot / 2]
  int64_t table;
  const void* positions;   // int32 or int64, [T] or [B][T], or null (0, 1, ..)
  int32_t positions64, per_batch;
  int32_t wtype;           // mscan_dtype of the weights
};

struct NormSide {          // queries or keys
  int32_t heads;
  Heads x, dy;
  const void* w;           // [D] or null (ones)
  void* y;                 // forward: the result; backward: dx. [B][T][heads][D]
};

void norm_bwd_blocks(const NormProblem& p, int Hq, int Hk, unsigned& qb, unsigned& kb);
// backward: partial holds D floats per workgroup (norm_bwd_blocks); dwq, dwk: [D] or null
hipError_t launch_norm(const NormProblem& p, const NormSide& q, const NormSide& k, int dtype, bool bwd, float* dwq,
                       float* dwk, float* partial, hipStream_t st);

}  // namespace la
}  // namespace mscan
