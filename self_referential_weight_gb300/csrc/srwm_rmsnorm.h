// srwm_rmsnorm.h -- host interface of the root-mean-square norm's kernels.
#pragma once

#include <cuda_runtime.h>

namespace srwm {

struct RmsParams {
    const void *x, *residual;    // [N, C]; residual or NULL.  Backward: x is the forward pass's sum
    const float* gamma;          // [C] or NULL (ones)
    void* y;                     // [N, C] of the input's type, or of e4m3
    float* scale;                // [N, C / block], e4m3 alone
    void* total;                 // [N, C]: x + residual, or NULL
    float* rstd;                 // [N]: written by the forward pass (or NULL), read by the backward pass
    const void *dy, *dtotal;     // [N, C]; dtotal or NULL
    void* dx;
    float* dgamma;               // [C] or NULL
    float* part;                 // workspace
    long long N;
    int C, block;                // block: channels of one scale
    float eps;
};

size_t rmsnorm_backward_scratch(long long N, int C);
int rmsnorm_launch(int dtype, int out, const RmsParams& p, cudaStream_t st);
int rmsnorm_backward_launch(int dtype, const RmsParams& p, cudaStream_t st);

}  // namespace srwm
