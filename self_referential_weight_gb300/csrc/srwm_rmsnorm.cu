// srwm_rmsnorm.cu -- root-mean-square norm of a row after the residual's
// addition, with the result in the input's type or in 8 bits with scales, and
// its gradients.
//
//   h = x + residual,  r = 1 / sqrt(mean(h^2) + eps),  y = h r gamma
//   e4m3: scale = max |y| / 448 over a block of channels, y8 = y / scale
//   d = dy gamma,  dx = dtotal + r (d - h r mean(d h r)),  dgamma = sum dy h r
// Memory bounds it: each row is read once and waits in registers for its sum of
// squares.  h enters the norm before it is rounded to its type on its way out.
// A row takes a warp where that is enough, else a CTA of up to 16, with one to four
// vectors a thread, all of whose loads are issued at once.  65536 rows of 1024
// channels in bf16 into 8 bits with scales of 128 channels take 73.4 us, 6.4 TB/s
// (0.95 of the copy rate); gradients of 65536 x 512 take 46 us and 5 for dgamma's
// partial sums.
#include <cuda_runtime.h>

#include <algorithm>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_rmsnorm.h"
#include "srwm_sum.h"
#include "srwm_vec.cuh"

namespace srwm {
namespace {

constexpr int kSms = 152;
constexpr int kMostThreads = 512;
constexpr float kE4m3Max = 448.f;

// The larger value, or NaN where one is (fmaxf would drop it).
__device__ __forceinline__ float max_nan(float a, float b)
{
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}

// The sum (or largest) over a row's threads: warps of one row, or one warp alone.
template <bool MAX>
__device__ __forceinline__ float row_join(float v, int warps, float* s)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        const float w = __shfl_xor_sync(0xffffffffu, v, o);
        v = MAX ? max_nan(v, w) : v + w;
    }
    if (warps == 1) return v;
    if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = v;
    __syncthreads();
    v = s[0];
    for (int i = 1; i < warps; ++i) v = MAX ? max_nan(v, s[i]) : v + s[i];
    __syncthreads();   // before s is used again
    return v;
}

// (a, b) as two e4m3 values, rounded to nearest even, past 448 to 448; a in the low byte.
__device__ __forceinline__ uint32_t e4m3_pair(float a, float b)
{
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(b), "f"(a));
    return r;
}

// top / 448 to the nearest, of a normal quotient (7 divides no nearest product's remainder so closely that one correction
// could miss), infinity or NaN.
__device__ __forceinline__ float e4m3_scale(float top)
{
    constexpr float kPart = 1.f / kE4m3Max;
    const float about = top * kPart;
    return isinf(about) ? about : fmaf(fmaf(-about, kE4m3Max, top), kPart, about);
}

// a / s to 24 bits, the last of them set where more follow (rounded to odd): a rounding to fewer bits is then the
// quotient's own.  One correction makes the product with inv = 1 / s the nearest value, whose remainder is exact; that
// gives the value towards zero and tells whether anything follows.
__device__ __forceinline__ float quotient_odd(float a, float s, float inv)
{
    const float about = a * inv;
    const float near = fmaf(fmaf(-about, s, a), inv, about);
    const float rest = fmaf(-near, s, a);
    const uint32_t q = __float_as_uint(__fmaf_rz(rest, inv, near));
    return __uint_as_float(rest != 0.f ? q | 1u : q);
}

// The e4m3 codes of v / s, to the nearest (ties to even).  A product with the approximate 1 / s is off by 2^-22 of itself at
// most; two of them, 2^-21 to either side, bracket the quotient, and where both give one code, that is it.  Only values
// next to a border between two codes are divided (65536 x 1024 bf16 73.0 us; all of them divided 80.3, products alone,
// which err there, 72.9).
template <int V>
__device__ __forceinline__ void e4m3_codes(const float (&v)[V], float s, uint32_t (&q)[V / 4])
{
    const float inv = s == 0.f ? 0.f : rcp_approx(s), less = inv * (1.f - 0x1p-21f), more = inv * (1.f + 0x1p-21f);
    bool same = true;
#pragma unroll
    for (int i = 0; i < V; i += 4) {
        q[i / 4] = e4m3_pair(v[i] * more, v[i + 1] * more) | e4m3_pair(v[i + 2] * more, v[i + 3] * more) << 16;
        same &= q[i / 4] == (e4m3_pair(v[i] * less, v[i + 1] * less) | e4m3_pair(v[i + 2] * less, v[i + 3] * less) << 16);
    }
    if (same) return;
    const float by = 1.f / s;
#pragma unroll
    for (int i = 0; i < V; i += 4)
        q[i / 4] = e4m3_pair(quotient_odd(v[i], s, by), quotient_odd(v[i + 1], s, by)) |
                   e4m3_pair(quotient_odd(v[i + 2], s, by), quotient_odd(v[i + 3], s, by)) << 16;
}

__device__ __forceinline__ void gamma_of(const RmsParams& p, int c, float (&g)[4])
{
    const float4 v = p.gamma ? __ldg(reinterpret_cast<const float4*>(p.gamma + c)) : make_float4(1.f, 1.f, 1.f, 1.f);
    g[0] = v.x, g[1] = v.y, g[2] = v.z, g[3] = v.w;
}
__device__ __forceinline__ void gamma_of(const RmsParams& p, int c, float (&g)[8])
{
    float a[4], b[4];
    gamma_of(p, c, a);
    gamma_of(p, c + 4, b);
#pragma unroll
    for (int k = 0; k < 4; ++k) g[k] = a[k], g[k + 4] = b[k];
}

enum Out { kSame, kE4m3Rows, kE4m3Blocks };   // a scale for a row, or for 128 channels

// warps: of a row; with one, a CTA's warps take a row each.
template <typename E, int K, int OUT>
__global__ void __launch_bounds__(kMostThreads) rms_kernel(const RmsParams p, int warps)
{
    constexpr int V = vec<E>;
    __shared__ float s[kMostThreads / 32];
    const int tpr = warps * 32;
    const long long row = warps == 1 ? static_cast<long long>(blockIdx.x) * (blockDim.x / 32) + (threadIdx.x >> 5) : blockIdx.x;
    if (row >= p.N) return;   // a whole warp, of a CTA whose warps do not meet
    const int at = warps == 1 ? threadIdx.x & 31 : threadIdx.x, nv = p.C / V;
    const size_t base = static_cast<size_t>(row) * p.C;
    uint4 rx[K], rr[K];
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at + k * tpr;
        if (v < nv) {
            rx[k] = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.x) + base + v * V);
            if (p.residual) rr[k] = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.residual) + base + v * V);
        }
    }
    float h[K][V], sq = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at + k * tpr;
        if (v < nv) {
            unpack(rx[k], h[k], E{});
            if (p.residual) {
                float r[V];
                unpack(rr[k], r, E{});
#pragma unroll
                for (int i = 0; i < V; ++i) h[k][i] += r[i];
            }
#pragma unroll
            for (int i = 0; i < V; ++i) sq = fmaf(h[k][i], h[k][i], sq);
            if (p.total) store_vec<E>(p.total, base + v * V, pack(h[k], E{}));
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) h[k][i] = 0.f;
        }
    }
    const float rstd = 1.f / sqrtf(row_join<false>(sq, warps, s) / p.C + p.eps);
    if (p.rstd && at == 0) p.rstd[row] = rstd;
    float top = 0.f;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at + k * tpr;
        if (v < nv) {
            float g[V];
            gamma_of(p, v * V, g);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                h[k][i] = h[k][i] * rstd * g[i];
                if (OUT == kE4m3Rows) top = max_nan(top, fabsf(h[k][i]));
            }
            if (OUT == kSame) store_vec<E>(p.y, base + v * V, pack(h[k], E{}));
        }
    }
    if constexpr (OUT != kSame) {
        if (OUT == kE4m3Rows) top = row_join<true>(top, warps, s);
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at + k * tpr;
            if constexpr (OUT == kE4m3Blocks) {   // 128 channels: as many neighbouring lanes as they have vectors
                top = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) top = max_nan(top, fabsf(h[k][i]));
#pragma unroll
                for (int o = 128 / V / 2; o > 0; o >>= 1) top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, o));
            }
            if (v >= nv) continue;
            // a block next to zero is lifted first: the quotients' remainders have to stay above fp32's smallest number
            float scale = e4m3_scale(top), by = scale;
            if (top < 0x1p-60f) {
                scale = top / kE4m3Max;
                by = e4m3_scale(top * 0x1p100f);
#pragma unroll
                for (int i = 0; i < V; ++i) h[k][i] *= 0x1p100f;
            }
            uint32_t q[V / 4];
            e4m3_codes(h[k], by, q);
            unsigned char* const to = static_cast<unsigned char*>(p.y) + base + v * V;
            if constexpr (V == 8)
                *reinterpret_cast<uint2*>(to) = make_uint2(q[0], q[1]);
            else
                *reinterpret_cast<uint32_t*>(to) = q[0];
            if (OUT == kE4m3Rows ? v == 0 : v % (128 / V) == 0)
                p.scale[OUT == kE4m3Rows ? row : row * (p.C / 128) + v / (128 / V)] = scale;
        }
    }
}

// Rows part, part + parts, ...: dx, and part [parts, C] of dgamma.
template <typename E, int K>
__global__ void __launch_bounds__(kMostThreads) rms_grad_kernel(const RmsParams p, int warps, int parts)
{
    constexpr int V = vec<E>;
    constexpr bool AHEAD = K < 4;     // the next row's loads are on their way while one is worked on: where registers hold both
    extern __shared__ float sums[];   // [rows of the CTA, C] where a warp takes a row
    __shared__ float s[kMostThreads / 32];
    const int tpr = warps * 32, rows = warps == 1 ? blockDim.x / 32 : 1;
    const int at = warps == 1 ? threadIdx.x & 31 : threadIdx.x, mine = warps == 1 ? threadIdx.x >> 5 : 0, nv = p.C / V;
    float dg[K][V];
#pragma unroll
    for (int k = 0; k < K; ++k)
#pragma unroll
        for (int i = 0; i < V; ++i) dg[k][i] = 0.f;
    const float inv = 1.f / p.C;
    struct Row {
        uint4 h[K], d[K], t[K];
        float rstd;
    };
    auto load = [&](long long row, Row& r) {
        const size_t base = static_cast<size_t>(row) * p.C;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at + k * tpr;
            if (v < nv) {
                r.h[k] = load_vec<E>(p.x, base + v * V);
                r.d[k] = load_vec<E>(p.dy, base + v * V);
                if (p.dtotal) r.t[k] = load_vec<E>(p.dtotal, base + v * V);
            }
        }
        r.rstd = __ldg(p.rstd + row);
    };
    const long long step = static_cast<long long>(parts) * rows;
    long long row = static_cast<long long>(blockIdx.x) * rows + mine;
    Row now, next;
    if (AHEAD && row < p.N) load(row, now);
    for (; row < p.N; row += step) {
        if (!AHEAD) load(row, now);
        if (AHEAD && row + step < p.N) load(row + step, next);
        const size_t base = static_cast<size_t>(row) * p.C;
        float xh[K][V], d[K][V], dot = 0.f;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at + k * tpr;
            if (v < nv) {
                float g[V];
                gamma_of(p, v * V, g);
                unpack(now.h[k], xh[k], E{});
                unpack(now.d[k], d[k], E{});
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    xh[k][i] *= now.rstd;
                    dg[k][i] = fmaf(d[k][i], xh[k][i], dg[k][i]);
                    d[k][i] *= g[i];
                    dot = fmaf(d[k][i], xh[k][i], dot);
                }
            }
        }
        const float m = row_join<false>(dot, warps, s) * inv;
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int v = at + k * tpr;
            if (v < nv) {
                float out[V];
                if (p.dtotal)
                    unpack(now.t[k], out, E{});
                else
#pragma unroll
                    for (int i = 0; i < V; ++i) out[i] = 0.f;
#pragma unroll
                for (int i = 0; i < V; ++i) out[i] = fmaf(now.rstd, fmaf(-xh[k][i], m, d[k][i]), out[i]);
                store_vec<E>(p.dx, base + v * V, pack(out, E{}));
            }
        }
        if (AHEAD) now = next;
    }
    griddep_launch();
    if (!p.part) return;
    float* const to = p.part + static_cast<size_t>(blockIdx.x) * p.C;
    float* const from = rows == 1 ? to : sums + static_cast<size_t>(mine) * p.C;
#pragma unroll
    for (int k = 0; k < K; ++k) {
        const int v = at + k * tpr;
        if (v < nv)
#pragma unroll
            for (int i = 0; i < V; i += 4)
                *reinterpret_cast<float4*>(from + v * V + i) = make_float4(dg[k][i], dg[k][i + 1], dg[k][i + 2], dg[k][i + 3]);
    }
    if (rows == 1) return;
    __syncthreads();
    for (int c = threadIdx.x; c < p.C; c += blockDim.x) {
        float a = 0.f;
        for (int r = 0; r < rows; ++r) a += sums[static_cast<size_t>(r) * p.C + c];
        to[c] = a;
    }
}

// Warps of a row and vectors of a thread: four vectors, or one (where 512 threads hold a row) while there are too few of them
// to fill the SMs.  One against four, 4096 channels in fp16: 96 rows 2.7 and 3.2 us, 300 3.2 and 3.6, 600 4.5 and 4.0; 1024
// channels in bf16: 600 rows 2.6 and 3.1, 2400 3.8 and 3.8.
struct RowPlan {
    int warps, vectors, rows;   // rows: of a CTA
};

RowPlan row_plan(size_t e, long long N, int C)
{
    const int nv = C / static_cast<int>(16 / e);
    RowPlan r{};
    r.vectors = nv <= 32 ? 1 : nv <= 64 ? 2 : 4;
    while (r.vectors > 1 && N * nv < (1 << 18) && (nv + r.vectors / 2 - 1) / (r.vectors / 2) <= kMostThreads) r.vectors /= 2;
    r.warps = ((nv + r.vectors - 1) / r.vectors + 31) / 32;
    r.rows = r.warps == 1 ? 4 : 1;
    return r;
}

// The gradients' rows take up to two vectors a thread where they fit (their partial sums stay in registers), and as many
// CTAs as run at once.
RowPlan grad_plan(size_t e, int C)
{
    const int nv = C / static_cast<int>(16 / e);
    RowPlan r{};
    r.vectors = nv <= 32 ? 1 : nv <= 2 * kMostThreads ? 2 : 4;
    r.warps = ((nv + r.vectors - 1) / r.vectors + 31) / 32;
    r.rows = r.warps == 1 ? 8 : 1;
    return r;
}

int grad_parts(const RowPlan& r, long long N)
{
    const long long most = kSms * std::max(1, 16 / (r.warps * r.rows));   // CTAs that share the SMs
    return static_cast<int>(std::max(1LL, std::min<long long>((N + r.rows - 1) / r.rows, most)));
}

template <typename E, int K>
int forward(const RmsParams& p, const RowPlan& r, int out, cudaStream_t st)
{
    const unsigned grid = static_cast<unsigned>((p.N + r.rows - 1) / r.rows);
    const int threads = 32 * r.warps * r.rows;
    if (!out)
        rms_kernel<E, K, kSame><<<grid, threads, 0, st>>>(p, r.warps);
    else if (p.block == 128 && p.C != 128)
        rms_kernel<E, K, kE4m3Blocks><<<grid, threads, 0, st>>>(p, r.warps);
    else
        rms_kernel<E, K, kE4m3Rows><<<grid, threads, 0, st>>>(p, r.warps);
    return launched();
}

template <typename E, int K>
int backward(const RmsParams& p0, const RowPlan& r, cudaStream_t st)
{
    RmsParams p = p0;
    if (!p.dgamma) p.part = nullptr;
    const int parts = grad_parts(r, p.N);
    const size_t smem = r.rows > 1 && p.part ? static_cast<size_t>(r.rows) * p.C * 4 : 0;   // a warp's row: at most 16 KB for eight
    rms_grad_kernel<E, K><<<parts, 32 * r.warps * r.rows, smem, st>>>(p, r.warps, parts);
    const int rc = launched();
    if (rc != SRWM_OK || !p.dgamma) return rc;
    return sum_launch({p.part, parts, {p.dgamma, nullptr, nullptr}, {p.C, 0, 0}, false}, st);
}

template <typename E>
int by_vectors(const RmsParams& p, int out, cudaStream_t st)
{
    const RowPlan r = row_plan(sizeof(E), p.N, p.C);
    return r.vectors == 1 ? forward<E, 1>(p, r, out, st) : r.vectors == 2 ? forward<E, 2>(p, r, out, st) : forward<E, 4>(p, r, out, st);
}

template <typename E>
int grad_by_vectors(const RmsParams& p, cudaStream_t st)
{
    const RowPlan r = grad_plan(sizeof(E), p.C);
    if constexpr (sizeof(E) == 4)
        if (r.vectors == 4) return backward<E, 4>(p, r, st);   // more than 4096 channels
    return r.vectors == 1 ? backward<E, 1>(p, r, st) : backward<E, 2>(p, r, st);
}

}  // namespace

size_t rmsnorm_backward_scratch(long long N, int C)
{
    const int parts = std::max(grad_parts(grad_plan(4, C), N), grad_parts(grad_plan(2, C), N));
    return round256(static_cast<size_t>(parts) * C * 4);
}

int rmsnorm_launch(int dtype, int out, const RmsParams& p, cudaStream_t st)
{
    if (p.N == 0) return SRWM_OK;
    if (dtype == SRWM_F32) return by_vectors<float>(p, out, st);
    if (dtype == SRWM_BF16) return by_vectors<__nv_bfloat16>(p, out, st);
    return by_vectors<__half>(p, out, st);
}

int rmsnorm_backward_launch(int dtype, const RmsParams& p, cudaStream_t st)
{
    if (dtype == SRWM_F32) return grad_by_vectors<float>(p, st);
    if (dtype == SRWM_BF16) return grad_by_vectors<__nv_bfloat16>(p, st);
    return grad_by_vectors<__half>(p, st);
}

}  // namespace srwm
