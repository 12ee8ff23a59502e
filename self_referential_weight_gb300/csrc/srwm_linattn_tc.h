// srwm_linattn_tc.h -- host interface of the tcgen05 kernel of the primitive in
// srwm_linattn.h (bf16, d = 64).
#pragma once

#include <cuda_runtime.h>

#include "srwm_linattn.h"

namespace srwm {

// Whether a call may take it: bf16, d = 64, an unsplit axis of at least one of its chunks.
bool linattn_tc_takes(int dtype, int d, const LinParams& p);
int linattn_tc_launch(int roles, const LinParams& p, cudaStream_t st);

}  // namespace srwm
