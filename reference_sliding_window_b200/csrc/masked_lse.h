// The masked forward that also leaves each row's log of its sum of exponentials,
// which the gradient recomputes the probabilities from.
#pragma once

#include "internal.h"

namespace rswa {

struct RowLse {
  float* lse;  // [H][stride] float32, natural log, or null
  int stride;
};
cudaError_t launch_masked_forward_simt(const MaskedParams& p, int elem, const RowLse& lse, cudaStream_t stream);
cudaError_t launch_masked_forward_tc(const MaskedParams& p, const RowLse& lse, cudaStream_t stream);

}  // namespace rswa
