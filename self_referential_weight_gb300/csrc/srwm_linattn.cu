// srwm_linattn.cu -- linear attention with a decay per head: the launches of
// the chunked kernel (srwm_linattn.cuh), and the single-token kernel.
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_linattn.cuh"
#include "srwm_linattn_scan.h"
#include "srwm_linattn_tc.h"

namespace srwm {
namespace {

constexpr int kMaxDevices = 64;

// Registers are capped so that this many CTAs share an SM; other counts measured slower or the same at D = 32 and 16.
template <typename E, int D>
constexpr int blocks_per_sm()
{
    return D == 64 ? 2 : D == 32 ? 4 : 10;
}

template <typename E, int D>
__global__ void __launch_bounds__(LinTile<E, D>::kThreads, blocks_per_sm<E, D>())
    linattn_kernel(const __grid_constant__ LinParams p)
{
    linattn_body<E, D, false>(p);
}

template <typename E, int D>
__global__ void __launch_bounds__(LinTile<E, D>::kThreads, blocks_per_sm<E, D>())
    linattn_state_kernel(const __grid_constant__ LinParams p)
{
    griddep_launch();
    linattn_body<E, D, true>(p);
}

// One token: S_out = g S_in + k v^T, o = scale S_out^T q.  Bound by the state,
// read and written once.  kWarps warps per stream; a lane holds float4 pieces
// of rows `stride` apart, all loaded before the first is used.  8192 states of
// d = 64 (268 MB in and out) take 41.5 us, 0.97 of the copy rate.
template <typename E, int D>
__global__ void __launch_bounds__(128) linattn_step_kernel(const E* __restrict__ q, const E* __restrict__ k,
                                                           const E* __restrict__ v, long long ld,
                                                           const float* __restrict__ log_decay, const float* S_in,
                                                           int streams, int H, float scale, E* __restrict__ o,
                                                           float* S_out)
{
    constexpr int kWarps = D == 64 ? 4 : 1, kStreams = 4 / kWarps, kCols = D / 4;   // float4 columns
    constexpr int stride = 32 * kWarps / kCols, kRows = D / stride;
    __shared__ float4 s_o[D == 64 ? 4 : 1][16];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int stream = blockIdx.x * kStreams + warp / kWarps;
    if (stream >= streams) return;   // whole warps, and only where a warp works alone
    const int b = stream / H, h = stream % H;
    const int t = (warp % kWarps) * 32 + lane, c = t % kCols, r0 = t / kCols;
    const size_t base = static_cast<size_t>(stream) * D * D;
    const float4* in = reinterpret_cast<const float4*>(S_in + base);
    float4 s[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) s[i] = in[(r0 + i * stride) * kCols + c];
    const long long row = b * ld + h * D;
    float qv[kRows], kv[kRows];
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        qv[i] = to_f(q[row + r0 + i * stride]);
        kv[i] = to_f(k[row + r0 + i * stride]);
    }
    const float4 vv = make_float4(to_f(v[row + 4 * c]), to_f(v[row + 4 * c + 1]), to_f(v[row + 4 * c + 2]),
                                  to_f(v[row + 4 * c + 3]));
    const Decay g = decay_over(decay_log2(log_decay[h]), 1);
    float4* out = reinterpret_cast<float4*>(S_out + base);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int i = 0; i < kRows; ++i) {
        float4 n;
        n.x = fmaf(s[i].x, g.m, fmaf(kv[i], vv.x, s[i].x * g.c));
        n.y = fmaf(s[i].y, g.m, fmaf(kv[i], vv.y, s[i].y * g.c));
        n.z = fmaf(s[i].z, g.m, fmaf(kv[i], vv.z, s[i].z * g.c));
        n.w = fmaf(s[i].w, g.m, fmaf(kv[i], vv.w, s[i].w * g.c));
        out[(r0 + i * stride) * kCols + c] = n;
        a.x = fmaf(qv[i], n.x, a.x);
        a.y = fmaf(qv[i], n.y, a.y);
        a.z = fmaf(qv[i], n.z, a.z);
        a.w = fmaf(qv[i], n.w, a.w);
    }
#pragma unroll
    for (int m = kCols; m < 32; m *= 2) {
        a.x += __shfl_xor_sync(0xffffffffu, a.x, m);
        a.y += __shfl_xor_sync(0xffffffffu, a.y, m);
        a.z += __shfl_xor_sync(0xffffffffu, a.z, m);
        a.w += __shfl_xor_sync(0xffffffffu, a.w, m);
    }
    if constexpr (kWarps > 1) {
        if (lane < kCols) s_o[warp][lane] = a;
        __syncthreads();
        if (warp != 0) return;
        a = s_o[0][lane % kCols];
#pragma unroll
        for (int w = 1; w < kWarps; ++w) {
            const float4 x = s_o[w][lane % kCols];
            a = make_float4(a.x + x.x, a.y + x.y, a.z + x.z, a.w + x.w);
        }
    }
    if (lane < kCols) {
        E* oo = o + static_cast<size_t>(stream) * D + 4 * lane;
        oo[0] = from_f<E>(scale * a.x);
        oo[1] = from_f<E>(scale * a.y);
        oo[2] = from_f<E>(scale * a.z);
        oo[3] = from_f<E>(scale * a.w);
    }
}

// Lets a kernel take more than 48 KB of shared memory, once per device.
int allow_smem(const void* kernel, int bytes, std::atomic<bool>* done)
{
    if (bytes <= 48 * 1024) return SRWM_OK;
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    if (done[dev].load()) return SRWM_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes) != cudaSuccess) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    done[dev].store(true);
    return SRWM_OK;
}

template <typename E, int D>
int launch(int roles, int slots, const LinParams& p, cudaStream_t st)
{
    using L = LinTile<E, D>;
    static std::atomic<bool> main_ok[kMaxDevices], state_ok[kMaxDevices];
    int rc = allow_smem(reinterpret_cast<const void*>(linattn_kernel<E, D>), L::kSmem, main_ok);
    if (rc != SRWM_OK) return rc;
    const unsigned streams = static_cast<unsigned>(p.B) * p.H;
    if (p.segments > 1) {
        rc = allow_smem(reinterpret_cast<const void*>(linattn_state_kernel<E, D>), L::kSmemState, state_ok);
        if (rc != SRWM_OK) return rc;
        linattn_state_kernel<E, D><<<dim3(streams * (p.segments - 1), slots), L::kThreads, L::kSmemState, st>>>(p);
        rc = launched();
        return rc != SRWM_OK ? rc
                             : launch_behind(linattn_kernel<E, D>, dim3(streams * p.segments, roles), L::kThreads,
                                             static_cast<int>(L::kSmem), st, p);
    }
    linattn_kernel<E, D><<<dim3(streams * p.segments, roles), L::kThreads, L::kSmem, st>>>(p);
    return launched();
}

template <typename E>
int by_width(int d, int roles, int slots, const LinParams& p, cudaStream_t st)
{
    if (d == 16) return launch<E, 16>(roles, slots, p, st);
    if (d == 32) return launch<E, 32>(roles, slots, p, st);
    return launch<E, 64>(roles, slots, p, st);
}

template <typename E>
int launch_step(int d, const void* q, const void* k, const void* v, long long ld, const float* lg, const float* S_in,
                int B, int H, float scale, void* o, float* S_out, cudaStream_t st)
{
    const int streams = B * H;
    const unsigned grid = d == 64 ? streams : (streams + 3) / 4;
    const E *qe = static_cast<const E*>(q), *ke = static_cast<const E*>(k), *ve = static_cast<const E*>(v);
    E* oe = static_cast<E*>(o);
    if (d == 16)
        linattn_step_kernel<E, 16><<<grid, 128, 0, st>>>(qe, ke, ve, ld, lg, S_in, streams, H, scale, oe, S_out);
    else if (d == 32)
        linattn_step_kernel<E, 32><<<grid, 128, 0, st>>>(qe, ke, ve, ld, lg, S_in, streams, H, scale, oe, S_out);
    else
        linattn_step_kernel<E, 64><<<grid, 128, 0, st>>>(qe, ke, ve, ld, lg, S_in, streams, H, scale, oe, S_out);
    return launched();
}

}  // namespace

LinPlan linattn_plan(int dtype, int B, int T, int H, int d, int roles)
{
    // CTAs that the GPU holds at once, about, at each width
    const long long slots = 152LL * (d == 64 ? 2 : d == 32 ? 4 : 10);
    const long long ctas = static_cast<long long>(B) * H * roles;
    const int chunks = T / d + (T % d != 0);
    const LinPlan whole{chunks > 0 ? chunks * d : d, 1};
    // Splitting fills the GPU when there are few streams, for a second pass over two of the three tensors.  A segment's
    // chunks and the states before it, which it adds up, both run one after another: 2 sqrt(chunks) segments are near
    // the best of both (16 streams of 1200 tokens, fp32, d = 32: 16.6 us with 19 segments, 21.5 with 4; 4 streams of
    // 8192, bf16, d = 16: 20.7 with 32, 23.7 with 64, 35.5 with 128).
    const double root = std::sqrt(static_cast<double>(chunks));
    long long segments = ctas * 3 > slots ? 1 : slots / ctas;
    segments = std::min(segments, static_cast<long long>(2 * root));
    if (segments < 2 || chunks < 8) return whole;   // below, the second launch costs what it saves
    if (d == 64 && dtype != SRWM_F16) {
        // Against that, the tcgen05 kernels take a whole stream's 128 tokens in 1.55 us (bf16) or 4.6 to 4.9 us (fp32)
        // however few streams there are; the split takes a time with the root of the chunks, and 2.0 or 3.6 us for each
        // stream's 8192 tokens (split and whole, fp32: 10 streams of 1200 23 and 50 us, 64 of 2500 89 and 96; bf16: 3 of
        // 1200 16 and 20, 16 of 2500 26 and 36, 32 of 8192 79 and 104).
        const bool wide = dtype == SRWM_F32;
        const double split = 6 + root * (wide ? 3.0 : 2.0) + static_cast<double>(ctas) * T * (wide ? 3.6 : 2.0) / 8192;
        if (split >= 5.0 + T / 128.0 * (wide ? 4.9 : 1.55)) return whole;
    }
    const int per = static_cast<int>((chunks + segments - 1) / segments);
    return {per * d, (chunks + per - 1) / per};
}

int linattn_launch(int dtype, int d, int roles, int slots, const LinParams& p, cudaStream_t st)
{
    if (linattn_scan_takes(dtype, d, roles, p)) return linattn_scan_launch(dtype, d, roles, p, st);
    if (linattn_tc_takes(dtype, d, p))
        return dtype == SRWM_F32 ? linattn_tc32_launch(roles, p, st) : linattn_tc_launch(roles, p, st);
    if (dtype == SRWM_F32) return by_width<float>(d, roles, slots, p, st);
    if (dtype == SRWM_BF16) return by_width<__nv_bfloat16>(d, roles, slots, p, st);
    return by_width<__half>(d, roles, slots, p, st);
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
