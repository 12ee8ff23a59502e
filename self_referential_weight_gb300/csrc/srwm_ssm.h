// srwm_ssm.h -- host interface of the selective state space scan's kernels.
#pragma once

#include <cuda_runtime.h>

namespace srwm {

struct SsmParams {
    const void *u, *dt, *z;                    // [B, T, D], token rows ld_u, ld_dt, ld_z elements apart; z or NULL
    const void *Bt, *Ct;                       // [B, T, G, N], token rows ld_bc elements apart
    const float *A, *skip, *dt_bias;           // [D, N]; [D] or NULL
    const float* h_in;                         // [B, D, N] or NULL (zeros)
    const int* lengths;                        // [B] or NULL
    void* y;                                   // [B, T, D]
    float* h_out;                              // [B, D, N] or NULL
    long long ld_u, ld_dt, ld_z, ld_bc;
    int B, T, D, N, G, softplus;
    // the first `whole` sequences run whole; the others' axis is cut into segments of seg_len tokens, whose own results
    // (from zero) are in the workspace.  first: of the blocks of all of these, the launch's first
    int whole, segments, seg_len, first;
    float *seg_state, *seg_dt;                 // [segments, B - whole, D, N], [segments, B - whole, D]
    // backward
    const void* dy;                            // [B, T, D]
    const float* dh_out;                       // [B, D, N] or NULL
    void *du, *ddt, *dz, *dB, *dC;             // du, ddt [B, T, D]; dz rows ld_dz, dB and dC rows ld_dbc elements apart
    long long ld_dz, ld_dbc;
    float *dA, *dskip, *ddt_bias, *dh_in;      // [D, N]; [D] or NULL; [B, D, N] or NULL
    float *seg_grad, *check, *bc_part, *part;  // workspace
    int base, span;                            // check, bc_part and part hold sequences base .. base + span - 1
    long long cut_row;                         // part's first row of the sequences that are cut
};

size_t ssm_scratch(int B, int T, int D, int N, int G);
size_t ssm_backward_scratch(int B, int T, int D, int N, int G);
int ssm_launch(int dtype, SsmParams& p, void* workspace, cudaStream_t st);
int ssm_step_launch(int dtype, const SsmParams& p, cudaStream_t st);
int ssm_backward_launch(int dtype, SsmParams& p, void* workspace, cudaStream_t st);

}  // namespace srwm
