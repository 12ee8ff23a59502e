// srwm_linattn_tc.h -- host interface of the tcgen05 kernels of the primitive in
// srwm_linattn.h (bf16 and fp32, d = 64).
#pragma once

#include <cuda_runtime.h>

#include "srwm_linattn.h"

namespace srwm {

// Whether a call may take them: an unsplit axis of at least one of their chunks.
bool linattn_tc_takes(int dtype, int d, const LinParams& p);
int linattn_tc_launch(int roles, const LinParams& p, cudaStream_t st);     // bf16
int linattn_tc32_launch(int roles, const LinParams& p, cudaStream_t st);   // fp32

}  // namespace srwm
