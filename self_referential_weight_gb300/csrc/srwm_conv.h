// srwm_conv.h -- host interface of the short causal convolution's kernels.
#pragma once

#include <cuda_runtime.h>

namespace srwm {

struct ConvParams {
    const void* x;               // [B, T, D], token rows ld elements apart
    long long ld;
    const float *weight, *bias;  // [D, W]; [D] or NULL
    const void* state_in;        // [B, W - 1, D] or NULL (zeros)
    const int* lengths;          // [B] or NULL
    const void *dy, *dstate;     // backward: [B, T, D]; [B, W - 1, D] or NULL
    void* y;                     // [B, T, D]
    void* state_out;             // [B, W - 1, D] or NULL; backward: dL/dstate_in
    void* dx;                    // [B, T, D], token rows ld_grad elements apart
    long long ld_grad;
    float *dweight, *dbias;      // [D, W] or NULL, [D] or NULL
    float* part;                 // workspace
    int B, T, D;
};

size_t conv_backward_scratch(int B, int T, int D, int W);
int conv_launch(int dtype, int W, int activation, const ConvParams& p, cudaStream_t st);
int conv_step_launch(int dtype, int W, int activation, const ConvParams& p, cudaStream_t st);
int conv_backward_launch(int dtype, int W, int activation, const ConvParams& p, cudaStream_t st);

}  // namespace srwm
