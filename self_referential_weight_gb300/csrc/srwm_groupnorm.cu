// srwm_groupnorm.cu -- group norm with an activation, channels last, and its
// gradients: one CTA per sample and group, one per channel for dgamma, dbeta.
#include <cuda_runtime.h>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_elem.cuh"
#include "srwm_groupnorm.h"

namespace srwm {
namespace {

constexpr int kThreads = 128;

template <int ACT>
__device__ __forceinline__ float act(float z)
{
    if constexpr (ACT == SRWM_ACT_SILU) return z / (1.f + expf(-z));
    if constexpr (ACT == SRWM_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    return z;
}

// Slope of the activation at z = xh * g + b, xh = (x - mean) * rstd.
template <int ACT>
__device__ __forceinline__ float slope(float x, float mean, float rstd, float g, float b)
{
    const float xh = (x - mean) * rstd, z = fmaf(xh, g, b);
    if constexpr (ACT == SRWM_ACT_SILU) {
        const float e = 1.f / (1.f + expf(-z));
        return e * fmaf(z, 1.f - e, 1.f);
    }
    if constexpr (ACT == SRWM_ACT_RELU) {
        // the side of the border decides a whole term of the gradient: within
        // fp32's error of it (a few roundings of both terms) it is taken in fp64
        if (fabsf(z) <= 1e-5f * (fabsf(x * rstd * g) + fabsf(mean * rstd * g) + fabsf(b))) {
            const double zd = (static_cast<double>(x) - mean) * rstd * g + b;
            return zd > 0.0 ? 1.f : 0.f;
        }
        return z > 0.f ? 1.f : 0.f;
    }
    return 1.f;
}

__device__ float block_sum(float v)
{
    __shared__ float s[kThreads];
    __syncthreads();
    s[threadIdx.x] = v;
    __syncthreads();
    for (int o = kThreads / 2; o > 0; o >>= 1) {
        if (threadIdx.x < o) s[threadIdx.x] += s[threadIdx.x + o];
        __syncthreads();
    }
    return s[0];
}

template <typename E, int ACT>
__global__ void __launch_bounds__(kThreads) gn_kernel(const GnParams p)
{
    const long long n = blockIdx.x;
    const int g = blockIdx.y, cg = p.C / p.G;
    const long long count = p.L * cg;
    const E* x = static_cast<const E*>(p.x) + n * p.L * p.C + g * cg;
    E* y = static_cast<E*>(p.y) + n * p.L * p.C + g * cg;
    float a = 0.f;
    for (long long i = threadIdx.x; i < count; i += kThreads) a += to_f(x[i / cg * p.C + i % cg]);
    const float mean = block_sum(a) / count;
    a = 0.f;
    for (long long i = threadIdx.x; i < count; i += kThreads) {
        const float d = to_f(x[i / cg * p.C + i % cg]) - mean;
        a = fmaf(d, d, a);
    }
    const float rstd = 1.f / sqrtf(block_sum(a) / count + p.eps);
    for (long long i = threadIdx.x; i < count; i += kThreads) {
        const int c = g * cg + i % cg;
        const float xh = (to_f(x[i / cg * p.C + i % cg]) - mean) * rstd;
        y[i / cg * p.C + i % cg] = from_f<E>(act<ACT>(fmaf(xh, p.gamma ? p.gamma[c] : 1.f, p.beta ? p.beta[c] : 0.f)));
    }
    if (threadIdx.x == 0) {
        if (p.mean) p.mean[n * p.G + g] = mean;
        if (p.rstd) p.rstd[n * p.G + g] = rstd;
    }
}

template <typename E, int ACT>
__global__ void __launch_bounds__(kThreads) gn_dx_kernel(const GnParams p)
{
    const long long n = blockIdx.x;
    const int g = blockIdx.y, cg = p.C / p.G;
    const long long count = p.L * cg, base = n * p.L * p.C + g * cg;
    const E *x = static_cast<const E*>(p.x) + base, *dy = static_cast<const E*>(p.dy) + base;
    E* dx = static_cast<E*>(p.dx) + base;
    const float mean = p.mean[n * p.G + g], rstd = p.rstd[n * p.G + g];
    float a = 0.f, b = 0.f;
    auto dh = [&](long long i, float* xh) {
        const int c = g * cg + i % cg;
        const float xv = to_f(x[i / cg * p.C + i % cg]), ga = p.gamma ? p.gamma[c] : 1.f;
        *xh = (xv - mean) * rstd;
        return to_f(dy[i / cg * p.C + i % cg]) * slope<ACT>(xv, mean, rstd, ga, p.beta ? p.beta[c] : 0.f) * ga;
    };
    for (long long i = threadIdx.x; i < count; i += kThreads) {
        float xh;
        const float v = dh(i, &xh);
        a += v;
        b = fmaf(v, xh, b);
    }
    a = block_sum(a) / count;
    b = block_sum(b) / count;
    for (long long i = threadIdx.x; i < count; i += kThreads) {
        float xh;
        const float v = dh(i, &xh);
        dx[i / cg * p.C + i % cg] = from_f<E>(rstd * (v - a - xh * b));
    }
}

template <typename E, int ACT>
__global__ void __launch_bounds__(kThreads) gn_dparam_kernel(const GnParams p)
{
    const int c = blockIdx.x, g = c / (p.C / p.G);
    const float ga = p.gamma ? p.gamma[c] : 1.f, be = p.beta ? p.beta[c] : 0.f;
    float a = 0.f, b = 0.f;
    for (long long i = threadIdx.x; i < p.N * p.L; i += kThreads) {
        const long long n = i / p.L;
        const float mean = p.mean[n * p.G + g], rstd = p.rstd[n * p.G + g];
        const float xv = to_f(static_cast<const E*>(p.x)[i * p.C + c]);
        const float dz = to_f(static_cast<const E*>(p.dy)[i * p.C + c]) * slope<ACT>(xv, mean, rstd, ga, be);
        a = fmaf(dz, (xv - mean) * rstd, a);
        b += dz;
    }
    a = block_sum(a);
    b = block_sum(b);
    if (threadIdx.x == 0) {
        if (p.dgamma) p.dgamma[c] = a;
        if (p.dbeta) p.dbeta[c] = b;
    }
}

template <typename E, int ACT>
int forward(const GnParams& p, cudaStream_t st)
{
    gn_kernel<E, ACT><<<dim3(static_cast<unsigned>(p.N), p.G), kThreads, 0, st>>>(p);
    return launched();
}

template <typename E, int ACT>
int backward(const GnParams& p, cudaStream_t st)
{
    if (p.N > 0) gn_dx_kernel<E, ACT><<<dim3(static_cast<unsigned>(p.N), p.G), kThreads, 0, st>>>(p);
    gn_dparam_kernel<E, ACT><<<p.C, kThreads, 0, st>>>(p);
    return launched();
}

template <typename E>
int by_act(bool back, int activation, const GnParams& p, cudaStream_t st)
{
    if (activation == SRWM_ACT_SILU)
        return back ? backward<E, SRWM_ACT_SILU>(p, st) : forward<E, SRWM_ACT_SILU>(p, st);
    if (activation == SRWM_ACT_RELU)
        return back ? backward<E, SRWM_ACT_RELU>(p, st) : forward<E, SRWM_ACT_RELU>(p, st);
    return back ? backward<E, SRWM_ACT_NONE>(p, st) : forward<E, SRWM_ACT_NONE>(p, st);
}

int by_type(bool back, int dtype, int activation, const GnParams& p, cudaStream_t st)
{
    if (dtype == SRWM_F32) return by_act<float>(back, activation, p, st);
    if (dtype == SRWM_BF16) return by_act<__nv_bfloat16>(back, activation, p, st);
    return by_act<__half>(back, activation, p, st);
}

}  // namespace

size_t groupnorm_scratch(long long, long long, int, int) { return 256; }
size_t groupnorm_backward_scratch(long long, long long, int, int) { return 256; }

int groupnorm_launch(int dtype, int activation, const GnParams& p, cudaStream_t st)
{
    return p.N == 0 ? SRWM_OK : by_type(false, dtype, activation, p, st);
}

int groupnorm_backward_launch(int dtype, int activation, const GnParams& p, cudaStream_t st)
{
    return by_type(true, dtype, activation, p, st);
}

}  // namespace srwm
