// srwm_linattn.cu -- linear attention with a decay per head: token-by-token
// kernels, one thread per state column.
#include <cuda_runtime.h>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_elem.cuh"
#include "srwm_linattn.h"

namespace srwm {
namespace {

__device__ __forceinline__ float decay_log2(float log_decay)
{
    return fmaxf(fminf(log_decay, 0.f) * 1.4426950408889634f, -16384.f);
}

template <typename E, int D>
__global__ void __launch_bounds__(D) linattn_kernel(const LinParams p)
{
    const LinRole& r = p.role[blockIdx.y];
    const int b = blockIdx.x / p.H, h = blockIdx.x % p.H, j = threadIdx.x;
    __shared__ float sa[D], sb[D];
    const float g = exp2f(decay_log2(p.log_decay[h]));
    const int n = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    float s[D];
    const size_t base = static_cast<size_t>(blockIdx.x) * D * D;
#pragma unroll
    for (int i = 0; i < D; ++i)
        s[i] = r.x_in ? r.x_in[base + (r.transposed ? j * D + i : i * D + j)] : 0.f;
    for (int i = 0; i < n; ++i) {
        const long long row = static_cast<long long>(b) * p.T + (r.reverse ? n - 1 - i : i);
        __syncthreads();
        sa[j] = to_f(static_cast<const E*>(r.a)[row * r.lda + h * D + j]);
        sb[j] = to_f(static_cast<const E*>(r.b)[row * r.ldb + h * D + j]);
        const float c = r.alpha_u * to_f(static_cast<const E*>(r.c)[row * r.ldc + h * D + j]);
        __syncthreads();
        float acc = 0.f;
#pragma unroll
        for (int k = 0; k < D; ++k) {
            s[k] = fmaf(sb[k], c, r.reverse ? s[k] : g * s[k]);
            acc = fmaf(sa[k], s[k], acc);
            if (r.reverse) s[k] *= g;
        }
        static_cast<E*>(r.out)[row * r.ldo + h * D + j] = from_f<E>(r.alpha_o * acc);
    }
    for (int t = n; t < p.T; ++t)
        static_cast<E*>(r.out)[(static_cast<long long>(b) * p.T + t) * r.ldo + h * D + j] = from_f<E>(0.f);
    if (r.x_out)
#pragma unroll
        for (int i = 0; i < D; ++i) r.x_out[base + (r.transposed ? j * D + i : i * D + j)] = s[i];
}

template <typename E, int D>
__global__ void __launch_bounds__(D) linattn_step_kernel(const E* q, const E* k, const E* v, long long ld,
                                                         const float* log_decay, const float* S_in, int H, float scale,
                                                         E* o, float* S_out)
{
    const int b = blockIdx.x / H, h = blockIdx.x % H, j = threadIdx.x;
    const float g = exp2f(decay_log2(log_decay[h]));
    const size_t base = static_cast<size_t>(blockIdx.x) * D * D;
    const long long row = b * ld + h * D;
    const float vj = to_f(v[row + j]);
    float acc = 0.f;
    for (int i = 0; i < D; ++i) {
        const float s = fmaf(to_f(k[row + i]), vj, g * S_in[base + i * D + j]);
        S_out[base + i * D + j] = s;
        acc = fmaf(to_f(q[row + i]), s, acc);
    }
    o[static_cast<size_t>(blockIdx.x) * D + j] = from_f<E>(scale * acc);
}

template <typename E>
int launch(int d, int roles, const LinParams& p, cudaStream_t st)
{
    const dim3 grid(static_cast<unsigned>(p.B) * p.H, roles);
    if (d == 16) linattn_kernel<E, 16><<<grid, 16, 0, st>>>(p);
    if (d == 32) linattn_kernel<E, 32><<<grid, 32, 0, st>>>(p);
    if (d == 64) linattn_kernel<E, 64><<<grid, 64, 0, st>>>(p);
    return launched();
}

template <typename E>
int launch_step(int d, const void* q, const void* k, const void* v, long long ld, const float* lg, const float* S_in,
                int B, int H, float scale, void* o, float* S_out, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>(B) * H;
    const E *qe = static_cast<const E*>(q), *ke = static_cast<const E*>(k), *ve = static_cast<const E*>(v);
    E* oe = static_cast<E*>(o);
    if (d == 16) linattn_step_kernel<E, 16><<<grid, 16, 0, st>>>(qe, ke, ve, ld, lg, S_in, H, scale, oe, S_out);
    if (d == 32) linattn_step_kernel<E, 32><<<grid, 32, 0, st>>>(qe, ke, ve, ld, lg, S_in, H, scale, oe, S_out);
    if (d == 64) linattn_step_kernel<E, 64><<<grid, 64, 0, st>>>(qe, ke, ve, ld, lg, S_in, H, scale, oe, S_out);
    return launched();
}

}  // namespace

int linattn_launch(int dtype, int d, int roles, const LinParams& p, cudaStream_t st)
{
    if (dtype == SRWM_F32) return launch<float>(d, roles, p, st);
    if (dtype == SRWM_BF16) return launch<__nv_bfloat16>(d, roles, p, st);
    return launch<__half>(d, roles, p, st);
}

int linattn_step_launch(int dtype, int d, const void* q, const void* k, const void* v, long long ld,
                        const float* log_decay, const float* S_in, int B, int H, float scale, void* o, float* S_out,
                        cudaStream_t st)
{
    if (dtype == SRWM_F32)
        return launch_step<float>(d, q, k, v, ld, log_decay, S_in, B, H, scale, o, S_out, st);
    if (dtype == SRWM_BF16)
        return launch_step<__nv_bfloat16>(d, q, k, v, ld, log_decay, S_in, B, H, scale, o, S_out, st);
    return launch_step<__half>(d, q, k, v, ld, log_decay, S_in, B, H, scale, o, S_out, st);
}

}  // namespace srwm
