// Rotary positions: the kernel's interface (the plan is rswa.h's rswa_rotary).
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

#include "internal.h"
#include "rswa.h"

namespace rswa {

// A [rows][heads][d] tensor and its result, rows `in_stride` / `out_stride`
// elements apart; in place when in == out.
struct RotaryTensor {
  const void* in;
  void* out;
  long long in_stride, out_stride;
  int heads;
};

struct RotaryParams {
  RotaryTensor x[2];         // queries, keys (heads = 0: none)
  const int32_t* positions;  // device [rows], or null
  int first;                 // without positions: row r is at first + r
  const int32_t* step_T;     // decode step of a handle: row b is at step_Lm[b] + step_T[0]
  const int32_t* step_Lm;
  int rows;
  float sign;                // -1: the inverse turn (the gradient)
  rswa_rotary plan;
};

cudaError_t launch_rotary(const RotaryParams& p, int elem, cudaStream_t stream);

}  // namespace rswa
