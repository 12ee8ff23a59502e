// srwm_ssm_api.cu -- the srwm_ssm_* entry points of include/srwm.h: argument
// checks and dispatch.
#include <cuda_runtime.h>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_ssm.h"

namespace {

using srwm::flat;
using srwm::Region;

bool sizes_ok(long long B, long long T, long long D, long long N, long long G)
{
    if (B <= 0 || T < 0 || D <= 0 || N <= 0 || G <= 0 || D % G != 0) return false;
    if (D > (1LL << 24) || B > (1LL << 30) / D || T > 0x3fffffffLL || G * N > (1LL << 30)) return false;
    return T == 0 || B * (D + 2 * G * N) <= (1LL << 40) / T;
}

bool supported(int D, int N, int G, int softplus)
{
    return D / G % 8 == 0 && (N == 16 || N == 32 || N == 64) && (softplus == 0 || softplus == 1);
}

bool ld_ok(long long ld, long long width, size_t e) { return ld >= width && ld <= (1LL << 40) && (static_cast<size_t>(ld) * e) % 16 == 0; }

Region rows_of(const void* p, long long n, long long ld, long long width, size_t e)
{
    return {p, static_cast<size_t>(width) * e, static_cast<size_t>(ld) * e, n};
}

}  // namespace

extern "C" {

size_t srwm_ssm_workspace_bytes(int B, int T, int D, int N, int G)
{
    return sizes_ok(B, T, D, N, G) && supported(D, N, G, 0) ? srwm::ssm_scratch(B, T, D, N, G) : 0;
}

size_t srwm_ssm_backward_workspace_bytes(int B, int T, int D, int N, int G)
{
    return sizes_ok(B, T, D, N, G) && supported(D, N, G, 0) ? srwm::ssm_backward_scratch(B, T, D, N, G) : 0;
}

int srwm_ssm_forward(const void* u, long long ld_u, const void* dt, long long ld_dt, const float* A, const void* Bt,
                     const void* Ct, long long ld_bc, const float* skip, const void* z, long long ld_z,
                     const float* dt_bias, int softplus, const float* h_init, const int* lengths, int dtype, int B, int T,
                     int D, int N, int G, void* y, float* h_final, void* workspace, size_t workspace_bytes, void* stream)
{
    if (!A || !workspace || (T > 0 && (!u || !dt || !Bt || !Ct || !y))) return SRWM_ERR_NULL;
    if (!sizes_ok(B, T, D, N, G)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(D, N, G, softplus) || e == 0) return SRWM_ERR_UNSUPPORTED;
    const long long gn = static_cast<long long>(G) * N, n = static_cast<long long>(B) * T;
    const size_t need = srwm::ssm_scratch(B, T, D, N, G);
    if (!ld_ok(ld_u, D, e) || !ld_ok(ld_dt, D, e) || (z && !ld_ok(ld_z, D, e)) || !ld_ok(ld_bc, gn, e) || workspace_bytes < need)
        return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({u, dt, A, Bt, Ct, skip, z, dt_bias, h_init, y, h_final, workspace});
    if (rc != SRWM_OK) return rc;
    if (reinterpret_cast<uintptr_t>(lengths) % 4 != 0) return SRWM_ERR_ALIGN;
    const size_t nd = static_cast<size_t>(D) * 4, state = static_cast<size_t>(B) * N * nd;
    rc = srwm::check_alias({rows_of(y, n, D, D, e), flat(h_final, state), flat(workspace, need)},
                           {rows_of(u, n, ld_u, D, e), rows_of(dt, n, ld_dt, D, e), rows_of(z, n, ld_z, D, e),
                            rows_of(Bt, n, ld_bc, gn, e), rows_of(Ct, n, ld_bc, gn, e), flat(A, nd * N), flat(skip, nd),
                            flat(dt_bias, nd), flat(h_init, state), flat(lengths, static_cast<size_t>(B) * 4)});
    if (rc != SRWM_OK) return rc;
    rc = T > 0 ? srwm::check_device_memory({u, dt, A, Bt, Ct, skip, z, dt_bias, h_init, lengths, y, h_final, workspace})
               : srwm::check_device_memory({A, skip, dt_bias, h_init, lengths, h_final, workspace});
    if (rc != SRWM_OK || (T == 0 && !h_final)) return rc;
    srwm::SsmParams p{};
    p.u = u, p.dt = dt, p.z = z, p.Bt = Bt, p.Ct = Ct, p.A = A, p.skip = skip, p.dt_bias = dt_bias, p.h_in = h_init;
    p.lengths = lengths, p.y = y, p.h_out = h_final;
    p.ld_u = ld_u, p.ld_dt = ld_dt, p.ld_z = ld_z, p.ld_bc = ld_bc;
    p.B = B, p.T = T, p.D = D, p.N = N, p.G = G, p.softplus = softplus;
    return srwm::ssm_launch(dtype, p, workspace, static_cast<cudaStream_t>(stream));
}

int srwm_ssm_step(const void* u, long long ld_u, const void* dt, long long ld_dt, const float* A, const void* Bt,
                  const void* Ct, long long ld_bc, const float* skip, const void* z, long long ld_z, const float* dt_bias,
                  int softplus, const float* h_in, int dtype, int B, int D, int N, int G, void* y, float* h_out, void* stream)
{
    if (!u || !dt || !A || !Bt || !Ct || !h_in || !y || !h_out) return SRWM_ERR_NULL;
    if (!sizes_ok(B, 1, D, N, G)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(D, N, G, softplus) || e == 0) return SRWM_ERR_UNSUPPORTED;
    const long long gn = static_cast<long long>(G) * N;
    if (!ld_ok(ld_u, D, e) || !ld_ok(ld_dt, D, e) || (z && !ld_ok(ld_z, D, e)) || !ld_ok(ld_bc, gn, e)) return SRWM_ERR_SHAPE;
    int rc = srwm::check_align({u, dt, A, Bt, Ct, skip, z, dt_bias, h_in, y, h_out});
    if (rc != SRWM_OK) return rc;
    const size_t nd = static_cast<size_t>(D) * 4, state = static_cast<size_t>(B) * N * nd;
    const Region hi = flat(h_out == h_in ? nullptr : h_in, state);   // exactly in place is allowed
    rc = srwm::check_alias({rows_of(y, B, D, D, e), flat(h_out, state)},
                           {rows_of(u, B, ld_u, D, e), rows_of(dt, B, ld_dt, D, e), rows_of(z, B, ld_z, D, e),
                            rows_of(Bt, B, ld_bc, gn, e), rows_of(Ct, B, ld_bc, gn, e), flat(A, nd * N), flat(skip, nd),
                            flat(dt_bias, nd), hi});
    if (rc != SRWM_OK) return rc;
    rc = srwm::check_device_memory({u, dt, A, Bt, Ct, skip, z, dt_bias, h_in, y, h_out});
    if (rc != SRWM_OK) return rc;
    srwm::SsmParams p{};
    p.u = u, p.dt = dt, p.z = z, p.Bt = Bt, p.Ct = Ct, p.A = A, p.skip = skip, p.dt_bias = dt_bias, p.h_in = h_in;
    p.y = y, p.h_out = h_out, p.ld_u = ld_u, p.ld_dt = ld_dt, p.ld_z = ld_z, p.ld_bc = ld_bc;
    p.B = B, p.T = 1, p.D = D, p.N = N, p.G = G, p.softplus = softplus;
    return srwm::ssm_step_launch(dtype, p, static_cast<cudaStream_t>(stream));
}

int srwm_ssm_backward(const void* u, long long ld_u, const void* dt, long long ld_dt, const float* A, const void* Bt,
                      const void* Ct, long long ld_bc, const float* skip, const void* z, long long ld_z,
                      const float* dt_bias, int softplus, const float* h_init, const int* lengths, int dtype, int B, int T,
                      int D, int N, int G, const void* dy, const float* dh_final, void* du, void* ddt, float* dA, void* dB,
                      void* dC, long long ld_dbc, float* dskip, void* dz, long long ld_dz, float* ddt_bias, float* dh_init,
                      void* workspace, size_t workspace_bytes, void* stream)
{
    if (!A || !dA || !workspace || (T > 0 && (!u || !dt || !Bt || !Ct || !dy || !du || !ddt || !dB || !dC || (z && !dz))))
        return SRWM_ERR_NULL;
    if (!sizes_ok(B, T, D, N, G)) return SRWM_ERR_SHAPE;
    const size_t e = srwm::dtype_bytes(dtype);
    if (!supported(D, N, G, softplus) || e == 0) return SRWM_ERR_UNSUPPORTED;
    const long long gn = static_cast<long long>(G) * N, n = static_cast<long long>(B) * T;
    const size_t need = srwm::ssm_backward_scratch(B, T, D, N, G);
    if (!ld_ok(ld_u, D, e) || !ld_ok(ld_dt, D, e) || (z && (!ld_ok(ld_z, D, e) || !ld_ok(ld_dz, D, e))) || !ld_ok(ld_bc, gn, e) ||
        !ld_ok(ld_dbc, gn, e) || workspace_bytes < need)
        return SRWM_ERR_SHAPE;
    if (!z) dz = nullptr;
    int rc = srwm::check_align({u, dt, A, Bt, Ct, skip, z, dt_bias, h_init, dy, dh_final, du, ddt, dA, dB, dC, dskip, dz,
                                ddt_bias, dh_init, workspace});
    if (rc != SRWM_OK) return rc;
    if (reinterpret_cast<uintptr_t>(lengths) % 4 != 0) return SRWM_ERR_ALIGN;
    const size_t nd = static_cast<size_t>(D) * 4, state = static_cast<size_t>(B) * N * nd;
    rc = srwm::check_alias({rows_of(du, n, D, D, e), rows_of(ddt, n, D, D, e), flat(dA, nd * N), rows_of(dB, n, ld_dbc, gn, e),
                            rows_of(dC, n, ld_dbc, gn, e), flat(dskip, nd), rows_of(dz, n, ld_dz, D, e), flat(ddt_bias, nd),
                            flat(dh_init, state), flat(workspace, need)},
                           {rows_of(u, n, ld_u, D, e), rows_of(dt, n, ld_dt, D, e), rows_of(z, n, ld_z, D, e),
                            rows_of(Bt, n, ld_bc, gn, e), rows_of(Ct, n, ld_bc, gn, e), flat(A, nd * N), flat(skip, nd),
                            flat(dt_bias, nd), flat(h_init, state), flat(lengths, static_cast<size_t>(B) * 4),
                            rows_of(dy, n, D, D, e), flat(dh_final, state)});
    if (rc != SRWM_OK) return rc;
    rc = T > 0 ? srwm::check_device_memory({u, dt, A, Bt, Ct, skip, z, dt_bias, h_init, lengths, dy, dh_final, du, ddt, dA, dB, dC,
                                            dskip, dz, ddt_bias, dh_init, workspace})
               : srwm::check_device_memory({A, skip, dt_bias, h_init, lengths, dh_final, dA, dskip, ddt_bias, dh_init, workspace});
    if (rc != SRWM_OK) return rc;
    srwm::SsmParams p{};
    p.u = u, p.dt = dt, p.z = z, p.Bt = Bt, p.Ct = Ct, p.A = A, p.skip = skip, p.dt_bias = dt_bias, p.h_in = h_init;
    p.lengths = lengths, p.ld_u = ld_u, p.ld_dt = ld_dt, p.ld_z = ld_z, p.ld_bc = ld_bc;
    p.B = B, p.T = T, p.D = D, p.N = N, p.G = G, p.softplus = softplus;
    p.dy = dy, p.dh_out = dh_final, p.du = du, p.ddt = ddt, p.dz = dz, p.dB = dB, p.dC = dC, p.ld_dz = ld_dz, p.ld_dbc = ld_dbc;
    p.dA = dA, p.dskip = dskip, p.ddt_bias = ddt_bias, p.dh_in = dh_init;
    return srwm::ssm_backward_launch(dtype, p, workspace, static_cast<cudaStream_t>(stream));
}

}  // extern "C"
