// srwm_linattn_api.cu -- the srwm_linattn_* entry points of include/srwm.h:
// argument checks, and each call as roles of the one primitive (srwm_linattn.h).
#include <cuda_runtime.h>

#include <cmath>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_linattn.h"

namespace {

using srwm::Region;

bool supported(int d) { return d == 16 || d == 32 || d == 64; }

bool sizes_ok(long long B, long long T, long long H, long long d)
{
    if (B <= 0 || H <= 0 || T < 0 || d <= 0) return false;
    return B * H <= 0x3fffffffLL && H * d <= 0x7fffffffLL && T <= 0x3fffffffLL && T <= (1LL << 46) / (B * H * d);
}

// A token-row array: rows of H * d elements, ld elements apart.
bool ld_ok(long long ld, long long H, long long d, size_t e)
{
    return ld >= H * d && ld <= (1LL << 40) && (static_cast<size_t>(ld) * e) % 16 == 0;
}

Region rows_of(const void* p, long long n, long long ld, long long H, long long d, size_t e)
{
    return {p, static_cast<size_t>(H * d) * e, static_cast<size_t>(ld) * e, n};
}

// Segment states, enough for any type (none when the axis is not split).
size_t scratch(int B, int T, int H, int d, int roles, int slots)
{
    size_t most = 256;
    for (int dtype : {SRWM_F32, SRWM_BF16, SRWM_F16}) {
        const srwm::LinPlan plan = srwm::linattn_plan(dtype, B, T, H, d, roles);
        const size_t need = static_cast<size_t>(slots) * plan.segments * B * H * d * d * 4;
        if (plan.segments > 1 && need > most) most = srwm::round256(need);
    }
    return most;
}

void set_plan(srwm::LinParams& p, int dtype, int d, int roles, void* workspace)
{
    const srwm::LinPlan plan = srwm::linattn_plan(dtype, p.B, p.T, p.H, d, roles);
    p.seg_len = plan.seg_len;
    p.segments = plan.segments;
    p.seg_state = static_cast<float*>(workspace);
}

}  // namespace

extern "C" {

size_t srwm_linattn_workspace_bytes(int B, int T, int H, int d)
{
    return sizes_ok(B, T, H, d) && supported(d) ? scratch(B, T, H, d, 1, 1) : 0;
}

size_t srwm_linattn_backward_workspace_bytes(int B, int T, int H, int d)
{
    return sizes_ok(B, T, H, d) && supported(d) ? scratch(B, T, H, d, 3, 2) : 0;
}

int srwm_linattn_forward(const void* q, const void* k, const void* v, long long ld, const float* log_decay,
                         const float* S_init, const int* lengths, int dtype, int B, int T, int H, int d,
                         float scale, void* o, float* S_final, void* workspace, size_t workspace_bytes,
                         void* stream)
{
    if (!log_decay || !workspace || (T > 0 && (!q || !k || !v || !o))) return SRWM_ERR_NULL;
    if (!sizes_ok(B, T, H, d)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(d) || e == 0) return SRWM_ERR_UNSUPPORTED;
    const size_t need = srwm_linattn_workspace_bytes(B, T, H, d);
    if (!ld_ok(ld, H, d, e) || workspace_bytes < need || !std::isfinite(scale)) return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({q, k, v, log_decay, S_init, o, S_final, workspace});
    if (rc != SRWM_OK) return rc;
    if (reinterpret_cast<uintptr_t>(lengths) % 4 != 0) return SRWM_ERR_ALIGN;
    const long long n = static_cast<long long>(B) * T;
    const size_t state = static_cast<size_t>(B) * H * d * d * 4;
    rc = srwm::check_alias({rows_of(o, n, static_cast<long long>(H) * d, H, d, e), srwm::flat(S_final, state),
                      srwm::flat(workspace, need)},
                     {rows_of(q, n, ld, H, d, e), rows_of(k, n, ld, H, d, e), rows_of(v, n, ld, H, d, e),
                      srwm::flat(log_decay, static_cast<size_t>(H) * 4), srwm::flat(S_init, state),
                      srwm::flat(lengths, static_cast<size_t>(B) * 4)});
    if (rc != SRWM_OK) return rc;
    rc = T > 0 ? srwm::check_device_memory({q, k, v, o, log_decay, S_init, lengths, S_final, workspace})
               : srwm::check_device_memory({log_decay, S_init, lengths, S_final, workspace});
    if (rc != SRWM_OK) return rc;
    srwm::LinParams p{};
    p.log_decay = log_decay;
    p.lengths = lengths;
    p.B = B, p.T = T, p.H = H;
    p.role[0] = {q, k, v, ld, ld, ld, o, static_cast<long long>(H) * d, S_init, S_final, 0, 0, 1.f, 0, scale, 0, 0};
    p.state_role[0] = 0;
    set_plan(p, dtype, d, 1, workspace);
    return srwm::linattn_launch(dtype, d, 1, 1, p, static_cast<cudaStream_t>(stream));
}

int srwm_linattn_step(const void* q, const void* k, const void* v, long long ld, const float* log_decay,
                      const float* S_in, int dtype, int B, int H, int d, float scale, void* o, float* S_out,
                      void* stream)
{
    if (!q || !k || !v || !log_decay || !S_in || !o || !S_out) return SRWM_ERR_NULL;
    if (!sizes_ok(B, 1, H, d)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(d) || e == 0) return SRWM_ERR_UNSUPPORTED;
    if (!ld_ok(ld, H, d, e) || !std::isfinite(scale)) return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({q, k, v, log_decay, S_in, o, S_out});
    if (rc != SRWM_OK) return rc;
    const size_t state = static_cast<size_t>(B) * H * d * d * 4;
    const Region si = srwm::flat(S_out == S_in ? nullptr : S_in, state);   // exactly in place is allowed
    rc = srwm::check_alias({rows_of(o, B, static_cast<long long>(H) * d, H, d, e), srwm::flat(S_out, state)},
                     {rows_of(q, B, ld, H, d, e), rows_of(k, B, ld, H, d, e), rows_of(v, B, ld, H, d, e),
                      srwm::flat(log_decay, static_cast<size_t>(H) * 4), si});
    if (rc != SRWM_OK) return rc;
    rc = srwm::check_device_memory({q, k, v, log_decay, S_in, o, S_out});
    if (rc != SRWM_OK) return rc;
    return srwm::linattn_step_launch(dtype, d, q, k, v, ld, log_decay, S_in, B, H, scale, o, S_out,
                                     static_cast<cudaStream_t>(stream));
}

int srwm_linattn_backward(const void* q, const void* k, const void* v, long long ld, const float* log_decay,
                          const float* S_init, const int* lengths, int dtype, int B, int T, int H, int d,
                          float scale, const void* do_, const float* dS_final, void* dq, void* dk, void* dv,
                          long long ld_grad, float* dS_init, void* workspace, size_t workspace_bytes,
                          void* stream)
{
    if (!log_decay || !workspace || (T > 0 && (!q || !k || !v || !do_ || !dq || !dk || !dv))) return SRWM_ERR_NULL;
    if (!sizes_ok(B, T, H, d)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(d) || e == 0) return SRWM_ERR_UNSUPPORTED;
    const size_t need = srwm_linattn_backward_workspace_bytes(B, T, H, d);
    if (!ld_ok(ld, H, d, e) || !ld_ok(ld_grad, H, d, e) || workspace_bytes < need || !std::isfinite(scale))
        return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({q, k, v, log_decay, S_init, do_, dS_final, dq, dk, dv, dS_init, workspace});
    if (rc != SRWM_OK) return rc;
    if (reinterpret_cast<uintptr_t>(lengths) % 4 != 0) return SRWM_ERR_ALIGN;
    const long long n = static_cast<long long>(B) * T, hd = static_cast<long long>(H) * d;
    const size_t state = static_cast<size_t>(B) * H * d * d * 4;
    rc = srwm::check_alias({rows_of(dq, n, ld_grad, H, d, e), rows_of(dk, n, ld_grad, H, d, e),
                      rows_of(dv, n, ld_grad, H, d, e), srwm::flat(dS_init, state), srwm::flat(workspace, need)},
                     {rows_of(q, n, ld, H, d, e), rows_of(k, n, ld, H, d, e), rows_of(v, n, ld, H, d, e),
                      rows_of(do_, n, hd, H, d, e), srwm::flat(log_decay, static_cast<size_t>(H) * 4),
                      srwm::flat(S_init, state), srwm::flat(dS_final, state),
                      srwm::flat(lengths, static_cast<size_t>(B) * 4)});
    if (rc != SRWM_OK) return rc;
    rc = T > 0 ? srwm::check_device_memory(
                     {q, k, v, do_, dq, dk, dv, log_decay, S_init, lengths, dS_final, dS_init, workspace})
               : srwm::check_device_memory({log_decay, S_init, lengths, dS_final, dS_init, workspace});
    if (rc != SRWM_OK) return rc;
    srwm::LinParams p{};
    p.log_decay = log_decay;
    p.lengths = lengths;
    p.B = B, p.T = T, p.H = H;
    // dq runs on S^T (from v and k), dv on D (from q and do), dk on D^T
    int ex = 0;
    const float man = 2.f * std::frexp(scale, &ex);
    p.role[0] = {do_, v, k, hd, ld, ld, dq, ld_grad, S_init, nullptr, 1, 0, 1.f, 0, scale, 0, 0};
    p.role[1] = {k, q, do_, ld, ld, hd, dv, ld_grad, dS_final, dS_init, 0, 1, man, ex - 1, 1.f, 1, 0};
    p.role[2] = {v, do_, q, ld, hd, ld, dk, ld_grad, dS_final, nullptr, 1, 1, man, ex - 1, 1.f, 1, 1};
    p.state_role[0] = 0;
    p.state_role[1] = 1;
    set_plan(p, dtype, d, 3, workspace);
    return srwm::linattn_launch(dtype, d, 3, 2, p,static_cast<cudaStream_t>(stream));
}

}  // extern "C"
