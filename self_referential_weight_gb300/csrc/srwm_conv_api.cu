// srwm_conv_api.cu -- the srwm_conv_* entry points of include/srwm.h: argument
// checks and dispatch.
#include <cuda_runtime.h>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_conv.h"

namespace {

using srwm::flat;
using srwm::Region;

bool sizes_ok(long long B, long long T, long long D)
{
    if (B <= 0 || T < 0 || D <= 0) return false;
    return B <= 0x3fffffffLL && T <= 0x3fffffffLL && D <= (1LL << 24) && B <= (1LL << 38) / D && (T == 0 || B * D <= (1LL << 42) / T);
}

bool supported(int D, int W, int activation)
{
    return D % 8 == 0 && W >= 2 && W <= 4 && (activation == SRWM_ACT_NONE || activation == SRWM_ACT_SILU);
}

bool ld_ok(long long ld, long long D, size_t e) { return ld >= D && ld <= (1LL << 40) && (static_cast<size_t>(ld) * e) % 16 == 0; }

Region rows_of(const void* p, long long n, long long ld, long long D, size_t e)
{
    return {p, static_cast<size_t>(D) * e, static_cast<size_t>(ld) * e, n};
}

}  // namespace

extern "C" {

size_t srwm_conv_backward_workspace_bytes(int B, int T, int D, int W)
{
    return sizes_ok(B, T, D) && supported(D, W, SRWM_ACT_NONE) ? srwm::conv_backward_scratch(B, T, D, W) : 0;
}

int srwm_conv_forward(const void* x, long long ld, const float* weight, const float* bias, const void* state_init,
                      const int* lengths, int dtype, int B, int T, int D, int W, int activation, void* y,
                      void* state_final, void* stream)
{
    if (!weight || (T > 0 && (!x || !y))) return SRWM_ERR_NULL;
    if (!sizes_ok(B, T, D)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(D, W, activation) || e == 0) return SRWM_ERR_UNSUPPORTED;
    if (!ld_ok(ld, D, e)) return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({x, weight, bias, state_init, y, state_final});
    if (rc != SRWM_OK) return rc;
    if (reinterpret_cast<uintptr_t>(lengths) % 4 != 0) return SRWM_ERR_ALIGN;
    const long long n = static_cast<long long>(B) * T;
    const size_t state = static_cast<size_t>(B) * (W - 1) * D * e, nd = static_cast<size_t>(D) * 4;
    rc = srwm::check_alias({rows_of(y, n, D, D, e), flat(state_final, state)},
                           {rows_of(x, n, ld, D, e), flat(weight, nd * W), flat(bias, nd), flat(state_init, state),
                            flat(lengths, static_cast<size_t>(B) * 4)});
    if (rc != SRWM_OK) return rc;
    rc = T > 0 ? srwm::check_device_memory({x, y, weight, bias, state_init, lengths, state_final})
               : srwm::check_device_memory({weight, bias, state_init, lengths, state_final});
    if (rc != SRWM_OK || (T == 0 && !state_final)) return rc;
    srwm::ConvParams p{};
    p.x = x, p.ld = ld, p.weight = weight, p.bias = bias, p.state_in = state_init, p.lengths = lengths;
    p.y = y, p.state_out = state_final, p.B = B, p.T = T, p.D = D;
    return srwm::conv_launch(dtype, W, activation, p, static_cast<cudaStream_t>(stream));
}

int srwm_conv_step(const void* x, long long ld, const float* weight, const float* bias, const void* state_in, int dtype,
                   int B, int D, int W, int activation, void* y, void* state_out, void* stream)
{
    if (!x || !weight || !state_in || !y || !state_out) return SRWM_ERR_NULL;
    if (!sizes_ok(B, 1, D)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(D, W, activation) || e == 0) return SRWM_ERR_UNSUPPORTED;
    if (!ld_ok(ld, D, e)) return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({x, weight, bias, state_in, y, state_out});
    if (rc != SRWM_OK) return rc;
    const size_t state = static_cast<size_t>(B) * (W - 1) * D * e, nd = static_cast<size_t>(D) * 4;
    const Region si = flat(state_out == state_in ? nullptr : state_in, state);   // exactly in place is allowed
    rc = srwm::check_alias({rows_of(y, B, D, D, e), flat(state_out, state)},
                           {rows_of(x, B, ld, D, e), flat(weight, nd * W), flat(bias, nd), si});
    if (rc != SRWM_OK) return rc;
    rc = srwm::check_device_memory({x, weight, bias, state_in, y, state_out});
    if (rc != SRWM_OK) return rc;
    srwm::ConvParams p{};
    p.x = x, p.ld = ld, p.weight = weight, p.bias = bias, p.state_in = state_in;
    p.y = y, p.state_out = state_out, p.B = B, p.T = 1, p.D = D;
    return srwm::conv_step_launch(dtype, W, activation, p, static_cast<cudaStream_t>(stream));
}

int srwm_conv_backward(const void* x, long long ld, const float* weight, const float* bias, const void* state_init,
                       const int* lengths, int dtype, int B, int T, int D, int W, int activation, const void* dy,
                       const void* dstate_final, void* dx, long long ld_grad, float* dweight, float* dbias,
                       void* dstate_init, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!weight || !workspace || (T > 0 && (!x || !dy || !dx))) return SRWM_ERR_NULL;
    if (!sizes_ok(B, T, D)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(D, W, activation) || e == 0) return SRWM_ERR_UNSUPPORTED;
    const size_t need = srwm::conv_backward_scratch(B, T, D, W);
    if (!ld_ok(ld, D, e) || !ld_ok(ld_grad, D, e) || workspace_bytes < need) return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({x, weight, bias, state_init, dy, dstate_final, dx, dweight, dbias, dstate_init, workspace});
    if (rc != SRWM_OK) return rc;
    if (reinterpret_cast<uintptr_t>(lengths) % 4 != 0) return SRWM_ERR_ALIGN;
    const long long n = static_cast<long long>(B) * T;
    const size_t state = static_cast<size_t>(B) * (W - 1) * D * e, nd = static_cast<size_t>(D) * 4;
    rc = srwm::check_alias({rows_of(dx, n, ld_grad, D, e), flat(dweight, nd * W), flat(dbias, nd), flat(dstate_init, state),
                            flat(workspace, need)},
                           {rows_of(x, n, ld, D, e), rows_of(dy, n, D, D, e), flat(weight, nd * W), flat(bias, nd),
                            flat(state_init, state), flat(dstate_final, state), flat(lengths, static_cast<size_t>(B) * 4)});
    if (rc != SRWM_OK) return rc;
    rc = T > 0 ? srwm::check_device_memory({x, dy, dx, weight, bias, state_init, lengths, dstate_final, dweight, dbias, dstate_init, workspace})
               : srwm::check_device_memory({weight, bias, state_init, lengths, dstate_final, dweight, dbias, dstate_init, workspace});
    if (rc != SRWM_OK) return rc;
    srwm::ConvParams p{};
    p.x = x, p.ld = ld, p.weight = weight, p.bias = bias, p.state_in = state_init, p.lengths = lengths;
    p.dy = dy, p.dstate = dstate_final, p.dx = dx, p.ld_grad = ld_grad, p.dweight = dweight, p.dbias = dbias;
    p.state_out = dstate_init, p.part = static_cast<float*>(workspace), p.B = B, p.T = T, p.D = D;
    return srwm::conv_backward_launch(dtype, W, activation, p, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
