// srwm_linattn.h -- the one primitive behind the linear attention entry points.
//
// With a decay g per head, processed positions i = 1 .. n of one stream and
// rows a_i, b_i, c_i:
//   H_i = X_{i-1} decayed + alpha_u b_i c_i^T,   out_i = alpha_o H_i^T a_i
// The forward pass and each of the three row gradients are this recurrence:
//   o  : a = q,  b = k,  c = v,  X = S                 tokens in order
//   dq : a = do, b = v,  c = k,  X = S^T               tokens in order
//   dv : a = k,  b = q,  c = do, X = D (dL/dS)         tokens in reverse
//   dk : a = v,  b = do, c = q,  X = D^T               tokens in reverse
// In order, the state decays before the token is added (S_t = g S_{t-1} + ...);
// in reverse it decays after (D_t = g D_{t+1} + ..., where the stored X is
// already g D_{t+1}), so that dS_final reaches the last token undecayed and
// the state left at the end is dS_init.
#pragma once

#include <cuda_runtime.h>

namespace srwm {

struct LinRole {
    const void *a, *b, *c;              // token rows, [B, T] rows of H * d elements
    long long lda, ldb, ldc;            // elements between two tokens' rows
    void* out;
    long long ldo;
    const float* x_in;                  // [B, H, d, d] or NULL (zero)
    float* x_out;                       // [B, H, d, d] or NULL
    int transposed;                     // x_in / x_out hold X^T
    int reverse;
    float alpha_u_man;                  // alpha_u = alpha_u_man * 2^alpha_u_exp, 1 <= |alpha_u_man| < 2 or 0
    int alpha_u_exp;
    float alpha_o;
    int state_slot;                     // whose segment states start this role's segments,
    int state_transposed;               // and whether they are X^T
};

struct LinParams {
    LinRole role[3];
    const float* log_decay;             // [H]
    const int* lengths;                 // [B] or NULL
    int B, T, H;
    // The long axis may be split into segments of seg_len positions (a multiple
    // of d).  The state each segment but the last adds is computed first, from
    // zero, by one pass for each of `slots` roles (state_role[slot]), into
    // seg_state [slots][segments][B * H][d * d] (the last segment's is unused);
    // then every segment starts from the decayed sum of the earlier ones'.
    int seg_len, segments;
    float* seg_state;
    int state_role[2];
};

// How a call of these sizes is split: segments and their length.  `roles` CTAs
// run per stream and segment (3 in the backward pass, 1 in the forward pass).
struct LinPlan {
    int seg_len, segments;
};
LinPlan linattn_plan(int dtype, int B, int T, int H, int d, int roles);

int linattn_launch(int dtype, int d, int roles, int slots, const LinParams& p, cudaStream_t st);
int linattn_step_launch(int dtype, int d, const void* q, const void* k, const void* v, long long ld,
                        const float* log_decay, const float* S_in, int B, int H, float scale, void* o, float* S_out,
                        cudaStream_t st);

}  // namespace srwm
