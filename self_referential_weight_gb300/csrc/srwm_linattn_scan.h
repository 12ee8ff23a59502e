// srwm_linattn_scan.h -- host interface of the token-by-token kernel of the
// primitive in srwm_linattn.h (short sequences).
#pragma once

#include <cuda_runtime.h>

#include "srwm_linattn.h"

namespace srwm {

bool linattn_scan_takes(int dtype, int d, int roles, const LinParams& p);
int linattn_scan_launch(int dtype, int d, int roles, const LinParams& p, cudaStream_t st);

}  // namespace srwm
