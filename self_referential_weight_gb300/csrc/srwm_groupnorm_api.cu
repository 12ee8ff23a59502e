// srwm_groupnorm_api.cu -- the srwm_groupnorm_* entry points of include/srwm.h:
// argument checks and dispatch.
#include <cuda_runtime.h>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_groupnorm.h"

namespace {

using srwm::flat;

constexpr int kMaxChannels = 8192;

int check_sizes(int dtype, long long N, long long L, int C, int G, int activation)
{
    if (N < 0 || L <= 0 || C <= 0 || G <= 0) return SRWM_ERR_SHAPE;
    if (N > 0x7fffffffLL || L > 0x7fffffffLL || (N > 0 && L > (1LL << 46) / N / C)) return SRWM_ERR_SHAPE;
    if (C % G != 0 || N * G > 0x7fffffffLL) return SRWM_ERR_SHAPE;
    if (C % 8 != 0 || C > kMaxChannels || srwm::dtype_bytes(dtype) == 0) return SRWM_ERR_UNSUPPORTED;
    if (activation != SRWM_ACT_NONE && activation != SRWM_ACT_SILU && activation != SRWM_ACT_RELU)
        return SRWM_ERR_UNSUPPORTED;
    return SRWM_OK;
}

}  // namespace

extern "C" {

size_t srwm_groupnorm_workspace_bytes(long long N, long long L, int C, int G)
{
    if (check_sizes(SRWM_F32, N, L, C, G, SRWM_ACT_NONE) != SRWM_OK) return 0;
    return srwm::groupnorm_scratch(N, L, C, G);
}

size_t srwm_groupnorm_backward_workspace_bytes(long long N, long long L, int C, int G)
{
    if (check_sizes(SRWM_F32, N, L, C, G, SRWM_ACT_NONE) != SRWM_OK) return 0;
    return srwm::groupnorm_backward_scratch(N, L, C, G);
}

int srwm_groupnorm_forward(const void* x, const float* gamma, const float* beta, int dtype, long long N,
                           long long L, int C, int G, float eps, int activation, void* y, float* mean,
                           float* rstd, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!workspace || (N > 0 && (!x || !y))) return SRWM_ERR_NULL;
    int rc = check_sizes(dtype, N, L, C, G, activation);
    if (rc != SRWM_OK) return rc;
    if (!(eps > 0.f)) return SRWM_ERR_UNSUPPORTED;
    const size_t need = srwm::groupnorm_scratch(N, L, C, G);
    if (workspace_bytes < need) return SRWM_ERR_SHAPE;
    for (const void* p : {x, static_cast<const void*>(gamma), static_cast<const void*>(beta),
                          static_cast<const void*>(y), static_cast<const void*>(mean),
                          static_cast<const void*>(rstd), static_cast<const void*>(workspace)})
        if (!srwm::aligned16(p)) return SRWM_ERR_ALIGN;
    const size_t nx = static_cast<size_t>(N) * L * C * srwm::dtype_bytes(dtype), nc = static_cast<size_t>(C) * 4;
    const size_t ns = static_cast<size_t>(N) * G * 4;
    const srwm::Region outs[] = {flat(y, nx), flat(mean, ns), flat(rstd, ns), flat(workspace, need)};
    const srwm::Region ins[] = {flat(x, nx), flat(gamma, nc), flat(beta, nc)};
    for (int i = 0; i < 4; ++i) {
        for (const auto& in : ins)
            if (srwm::overlap(outs[i], in)) return SRWM_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (srwm::overlap(outs[i], outs[j])) return SRWM_ERR_ALIAS;
    }
    if (N == 0) return SRWM_OK;
    rc = srwm::check_device_memory({x, y, gamma, beta, mean, rstd, workspace});
    if (rc != SRWM_OK) return rc;
    srwm::GnParams p{};
    p.x = x, p.gamma = gamma, p.beta = beta, p.y = y, p.mean = mean, p.rstd = rstd;
    p.part = static_cast<float*>(workspace);
    p.N = N, p.L = L, p.C = C, p.G = G, p.eps = eps;
    return srwm::groupnorm_launch(dtype, activation, p, static_cast<cudaStream_t>(stream));
}

int srwm_groupnorm_backward(const void* x, const float* gamma, const float* beta, const float* mean,
                            const float* rstd, const void* dy, int dtype, long long N, long long L, int C, int G,
                            int activation, void* dx, float* dgamma, float* dbeta, void* workspace,
                            size_t workspace_bytes, void* stream)
{
    if (!workspace || (N > 0 && (!x || !mean || !rstd || !dy || !dx))) return SRWM_ERR_NULL;
    int rc = check_sizes(dtype, N, L, C, G, activation);
    if (rc != SRWM_OK) return rc;
    const size_t need = srwm::groupnorm_backward_scratch(N, L, C, G);
    if (workspace_bytes < need) return SRWM_ERR_SHAPE;
    for (const void* p : {x, static_cast<const void*>(gamma), static_cast<const void*>(beta),
                          static_cast<const void*>(mean), static_cast<const void*>(rstd), dy,
                          static_cast<const void*>(dx), static_cast<const void*>(dgamma),
                          static_cast<const void*>(dbeta), static_cast<const void*>(workspace)})
        if (!srwm::aligned16(p)) return SRWM_ERR_ALIGN;
    const size_t nx = static_cast<size_t>(N) * L * C * srwm::dtype_bytes(dtype), nc = static_cast<size_t>(C) * 4;
    const size_t ns = static_cast<size_t>(N) * G * 4;
    const srwm::Region outs[] = {flat(dx, nx), flat(dgamma, nc), flat(dbeta, nc), flat(workspace, need)};
    const srwm::Region ins[] = {flat(x, nx), flat(dy, nx), flat(gamma, nc), flat(beta, nc), flat(mean, ns),
                                flat(rstd, ns)};
    for (int i = 0; i < 4; ++i) {
        for (const auto& in : ins)
            if (srwm::overlap(outs[i], in)) return SRWM_ERR_ALIAS;
        for (int j = i + 1; j < 4; ++j)
            if (srwm::overlap(outs[i], outs[j])) return SRWM_ERR_ALIAS;
    }
    rc = N > 0 ? srwm::check_device_memory({x, dy, dx, gamma, beta, mean, rstd, dgamma, dbeta, workspace})
               : srwm::check_device_memory({gamma, beta, dgamma, dbeta, workspace});
    if (rc != SRWM_OK) return rc;
    srwm::GnParams p{};
    p.x = x, p.dy = dy, p.gamma = gamma, p.beta = beta, p.dx = dx;
    p.mean = const_cast<float*>(mean), p.rstd = const_cast<float*>(rstd);
    p.dgamma = dgamma, p.dbeta = dbeta;
    p.part = static_cast<float*>(workspace);
    p.N = N, p.L = L, p.C = C, p.G = G;
    return srwm::groupnorm_backward_launch(dtype, activation, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
