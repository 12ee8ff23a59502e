// srwm_rmsnorm_api.cu -- the srwm_rmsnorm_* entry points of include/srwm.h:
// argument checks and dispatch.
#include <cuda_runtime.h>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_rmsnorm.h"

namespace {

using srwm::flat;

constexpr int kMaxChannels = 8192;

int check_sizes(int dtype, long long N, int C)
{
    if (N < 0 || C <= 0 || N > 0x7fffffffLL) return SRWM_ERR_SHAPE;
    return C % 8 != 0 || C > kMaxChannels || srwm::dtype_bytes(dtype) == 0 ? SRWM_ERR_UNSUPPORTED : SRWM_OK;
}

}  // namespace

extern "C" {

int srwm_rmsnorm_forward(const void* x, const void* residual, const float* gamma, int dtype, long long N, int C, float eps,
                         int out, int block, void* y, float* scale, void* total, float* rstd, void* stream)
{
    if (N > 0 && (!x || !y || (out == SRWM_OUT_E4M3 && !scale))) return SRWM_ERR_NULL;
    int rc = check_sizes(dtype, N, C);
    if (rc != SRWM_OK) return rc;
    if (!(eps > 0.f) || (out != SRWM_OUT_SAME && out != SRWM_OUT_E4M3)) return SRWM_ERR_UNSUPPORTED;
    if (out == SRWM_OUT_E4M3 ? block != 0 && block != 128 : block != 0) return SRWM_ERR_UNSUPPORTED;
    if (block == 128 && C % 128 != 0) return SRWM_ERR_SHAPE;
    rc = srwm::check_align({x, residual, gamma, y, scale, total, rstd});
    if (rc != SRWM_OK) return rc;
    const size_t n = static_cast<size_t>(N) * C, nx = n * srwm::dtype_bytes(dtype), ns = static_cast<size_t>(N) * 4;
    const bool e4m3 = out == SRWM_OUT_E4M3;
    // the residual stream may be updated in place
    rc = srwm::check_alias({flat(y, e4m3 ? n : nx), flat(e4m3 ? scale : nullptr, ns * (block ? C / block : 1)), flat(total, nx), flat(rstd, ns)},
                           {flat(x, nx), flat(residual == total ? nullptr : residual, nx), flat(gamma, static_cast<size_t>(C) * 4)});
    if (rc != SRWM_OK || N == 0) return rc;
    rc = srwm::check_device_memory({x, residual, gamma, y, e4m3 ? scale : nullptr, total, rstd});
    if (rc != SRWM_OK) return rc;
    srwm::RmsParams p{};
    p.x = x, p.residual = residual, p.gamma = gamma, p.y = y, p.scale = scale, p.total = total, p.rstd = rstd;
    p.N = N, p.C = C, p.block = block ? block : C, p.eps = eps;
    return srwm::rmsnorm_launch(dtype, e4m3, p, static_cast<cudaStream_t>(stream));
}

size_t srwm_rmsnorm_backward_workspace_bytes(long long N, int C)
{
    return check_sizes(SRWM_F32, N, C) == SRWM_OK ? srwm::rmsnorm_backward_scratch(N, C) : 0;
}

int srwm_rmsnorm_backward(const void* total, const float* gamma, const float* rstd, const void* dy, const void* dtotal,
                          int dtype, long long N, int C, void* dx, float* dgamma, void* workspace, size_t workspace_bytes,
                          void* stream)
{
    if (!workspace || (N > 0 && (!total || !rstd || !dy || !dx))) return SRWM_ERR_NULL;
    int rc = check_sizes(dtype, N, C);
    if (rc != SRWM_OK) return rc;
    const size_t need = srwm::rmsnorm_backward_scratch(N, C);
    if (workspace_bytes < need) return SRWM_ERR_SHAPE;
    rc = srwm::check_align({total, gamma, rstd, dy, dtotal, dx, dgamma, workspace});
    if (rc != SRWM_OK) return rc;
    const size_t nx = static_cast<size_t>(N) * C * srwm::dtype_bytes(dtype), nc = static_cast<size_t>(C) * 4;
    rc = srwm::check_alias({flat(dx, nx), flat(dgamma, nc), flat(workspace, need)},
                           {flat(total, nx), flat(dy, nx), flat(dtotal, nx), flat(gamma, nc), flat(rstd, static_cast<size_t>(N) * 4)});
    if (rc != SRWM_OK) return rc;
    rc = N > 0 ? srwm::check_device_memory({total, gamma, rstd, dy, dtotal, dx, dgamma, workspace})
               : srwm::check_device_memory({gamma, dgamma, workspace});
    if (rc != SRWM_OK) return rc;
    srwm::RmsParams p{};
    p.x = total, p.gamma = gamma, p.rstd = const_cast<float*>(rstd), p.dy = dy, p.dtotal = dtotal, p.dx = dx;
    p.dgamma = dgamma, p.part = static_cast<float*>(workspace), p.N = N, p.C = C, p.block = C;
    return srwm::rmsnorm_backward_launch(dtype, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
