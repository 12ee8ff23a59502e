// srwm_groupnorm.h -- host interface of the group norm kernels.
#pragma once

#include <cuda_runtime.h>

namespace srwm {

struct GnParams {
    const void *x, *dy;
    const float *gamma, *beta;          // [C] or NULL (ones, zeros)
    void *y, *dx;
    float *mean, *rstd;                 // [N, G]: written by the forward pass (or NULL), read by the backward pass
    float *dgamma, *dbeta;              // [C] or NULL
    float* part;                        // workspace
    long long N, L;
    int C, G;
    float eps;
};

size_t groupnorm_scratch(long long N, long long L, int C, int G);
size_t groupnorm_backward_scratch(long long N, long long L, int C, int G);
int groupnorm_launch(int dtype, int activation, const GnParams& p, cudaStream_t st);
int groupnorm_backward_launch(int dtype, int activation, const GnParams& p, cudaStream_t st);

}  // namespace srwm
