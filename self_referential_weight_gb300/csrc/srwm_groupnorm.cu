// srwm_groupnorm.cu -- group norm with an activation, channels last, and its
// gradients.
//
//   xh = (x - mean) rstd,  z = xh gamma + beta,  y = act(z)
//   dz = dy act'(z),  A_c = sum dz,  B_c = sum dz xh  (over a sample's positions)
//   dx = rstd (dz gamma - m1 - xh m2),  m1 = mean of dz gamma over the group
//      = sum_c gamma_c A_c / count,  m2 = sum_c gamma_c B_c / count
//   dbeta_c, dgamma_c = sums of A_c, B_c over the samples
// Everything here is bound by memory: x (and dy) is to be read once and y (dx)
// written once.  What differs with the shape is where a group's values wait for
// their statistics, so there are four ways (gn_plan):
//   rows   L = 1 and a group of up to 32 whole 16-byte vectors: one vector per
//          thread in registers, statistics by shuffles.
//   line   L = 1 otherwise: one warp per group, its values re-read from L1.
//   slab   a cluster of up to 8 CTAs holds a sample (or some of its groups) in
//          shared memory, a range of positions each; statistics are exchanged
//          through distributed shared memory.
//   split  larger samples: per-channel statistics of ranges of positions to
//          scratch, a merge per group, and a second read of x (and dy).
// A thread keeps one vector of channels throughout, so per-channel values
// (gamma, beta, statistics, gradient sums) stay in registers.  All sums run in
// a fixed order.  Variances are of deviations from a mean (two passes where the
// values are at hand, else Welford's update), merged pairwise by
//   mean = m_a + d n_b / n,  M2 = M2_a + M2_b + d^2 n_a n_b / n,  d = m_b - m_a.
#include <cooperative_groups.h>
#include <cuda_runtime.h>

#include <algorithm>
#include <atomic>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_elem.cuh"
#include "srwm_f2.cuh"
#include "srwm_groupnorm.h"
#include "srwm_mma.cuh"
#include "srwm_ptx.cuh"
#include "srwm_vec.cuh"

namespace cg = cooperative_groups;

namespace srwm {
namespace {

constexpr int kMaxDevices = 64;
constexpr int kSms = 152;
constexpr int kMaxCluster = 8;
constexpr int kRowThreads = 256;
constexpr int kSmemMost = 227 * 1024;    // of a CTA
constexpr int kSmemPair = 112 * 1024;    // of each of two
constexpr int kSlabGood = 48 * 1024;     // with this many, four CTAs share an SM and their loads overlap

// ---------------------------------------------------------------- activation
template <int ACT>
__device__ __forceinline__ float act(float z)
{
    if constexpr (ACT == SRWM_ACT_SILU) return z * sigmoid(z);
    if constexpr (ACT == SRWM_ACT_RELU) return z > 0.f ? z : (z != z ? z : 0.f);
    return z;
}

// Two activations at once.
template <int ACT>
__device__ __forceinline__ float2 act2(float2 z)
{
    if constexpr (ACT == SRWM_ACT_SILU) {
        float2 e = mul2(both(-1.4426950408889634f), z);
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.x) : "f"(e.x));
        asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e.y) : "f"(e.y));
        e = add2(both(1.f), e);
        return mul2(z, make_float2(rcp_approx(e.x), rcp_approx(e.y)));
    }
    return make_float2(act<ACT>(z.x), act<ACT>(z.y));
}

// (x - mean) rstd g + b in pairs of fp32: each rounding's error is kept as a second number (Knuth's sum of two
// numbers with its error; a product's error by fma).
__device__ __noinline__ float border(float x, float mean, float rstd, float g, float b)
{
    auto sum = [](float u, float v, float& err) {
        const float s = __fadd_rn(u, v), w = __fsub_rn(s, u);
        err = __fadd_rn(__fsub_rn(u, __fsub_rn(s, w)), __fsub_rn(v, w));
        return s;
    };
    float dl, sl;
    const float d = sum(x, -mean, dl), r = __fmul_rn(rstd, g), rl = __fmaf_rn(rstd, g, -r);
    const float m = __fmul_rn(d, r), ml = __fmaf_rn(d, r, -m), s = sum(m, b, sl);
    return __fadd_rn(s, __fadd_rn(sl, __fadd_rn(ml, __fmaf_rn(d, rl, __fmul_rn(dl, r)))));
}

// Slope of the activation at z = (x - mean) rstd g + b.
template <int ACT>
__device__ __forceinline__ float slope(float x, float mean, float rstd, float g, float b, float xh)
{
    if constexpr (ACT == SRWM_ACT_SILU) {
        const float z = fmaf(xh, g, b);
        const float e = sigmoid(z);
        return e * fmaf(z, 1.f - e, 1.f);
    }
    if constexpr (ACT == SRWM_ACT_RELU) {
        float z = fmaf(xh, g, b);
        // the side of the border decides a whole term of the gradient: within fp32's error of it (a few roundings of
        // both terms) z is taken again from exact differences and products, good to 2^-45 of its terms.  fp64 would
        // do, but the compiler computes both sides of a condition this short, and fp64 is slow: 31.7M values of
        // fp16 took 717 us.
        if (fabsf(z) <= 1e-6f * (fabsf(x * rstd * g) + fabsf(mean * rstd * g) + fabsf(b))) z = border(x, mean, rstd, g, b);
        return z > 0.f ? 1.f : 0.f;
    }
    return 1.f;
}

// ---------------------------------------------------------------- statistics
struct Stat {
    float n, mean, m2;
};
__device__ __forceinline__ Stat merge(const Stat& a, const Stat& b)
{
    if (b.n == 0.f) return a;
    if (a.n == 0.f) return b;
    const float n = a.n + b.n, d = b.mean - a.mean, f = b.n / n;
    return {n, fmaf(d, f, a.mean), a.m2 + fmaf(d * d, a.n * f, b.m2)};
}

__device__ __forceinline__ float warp_sum(float v)
{
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
    return v;
}

// Sums over aligned sets of `lanes` neighbouring lanes, lanes a power of two.
template <int U>
__device__ __forceinline__ void lanes_sum(float (&v)[U], int lanes)
{
    for (int o = lanes >> 1; o > 0; o >>= 1)
#pragma unroll
        for (int u = 0; u < U; ++u) v[u] += __shfl_xor_sync(0xffffffffu, v[u], o);
}

template <int V>
struct Channels {   // per-channel values of a thread's vector
    float gamma[V], beta[V];
    __device__ __forceinline__ Channels(const GnParams& p, int c)
    {
#pragma unroll
        for (int k = 0; k < V; k += 4) {
            const float4 g = p.gamma ? __ldg(reinterpret_cast<const float4*>(p.gamma + c + k)) : make_float4(1.f, 1.f, 1.f, 1.f);
            const float4 b = p.beta ? __ldg(reinterpret_cast<const float4*>(p.beta + c + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
            gamma[k] = g.x, gamma[k + 1] = g.y, gamma[k + 2] = g.z, gamma[k + 3] = g.w;
            beta[k] = b.x, beta[k + 1] = b.y, beta[k + 2] = b.z, beta[k + 3] = b.w;
        }
    }
};

// ---------------------------------------------------------------- rows
// Block of kRowThreads: `slots` rows of `tile` vectors.  A thread's rows are
// `slots` * gridDim.x apart; U of them are in flight at once.
struct RowTile {
    int tile, slots, lanes, vecs;   // lanes of one group, and the vectors that they hold (idle lanes fill up to a power of two)
};
template <typename E>
__host__ __device__ RowTile row_tile(int C, int G)
{
    RowTile t;
    t.vecs = C / G / vec<E>;
    t.lanes = 1;
    while (t.lanes < t.vecs) t.lanes *= 2;
    const int cv = G * t.lanes;
    t.tile = cv < kRowThreads ? cv : kRowThreads;
    t.slots = kRowThreads / t.tile;
    return t;
}

template <typename E, int ACT, int U>
__global__ void __launch_bounds__(kRowThreads, 3) gn_rows_kernel(const GnParams p)
{
    constexpr int V = vec<E>;
    const RowTile rt = row_tile<E>(p.C, p.G);
    const int slot = threadIdx.x / rt.tile, v = blockIdx.y * kRowThreads + threadIdx.x % rt.tile;
    const int group = v / rt.lanes, c = (group * rt.vecs + v % rt.lanes) * V;
    const bool on = slot < rt.slots && group < p.G && v % rt.lanes < rt.vecs;
    const Channels<V> ch(p, on ? c : 0);
    const float inv = 1.f / static_cast<float>(rt.vecs * V);
    const long long step = static_cast<long long>(gridDim.x) * rt.slots;
    for (long long base = static_cast<long long>(blockIdx.x) * rt.slots; base < p.N; base += step * U) {
        float x[U][V], sum[U], sq[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = base + u * step + slot;
            unpack(on && row < p.N ? load_vec<E>(p.x, static_cast<size_t>(row) * p.C + c) : make_uint4(0, 0, 0, 0), x[u],
                   E{});
        }
        auto pair = [&x](int u, int k) { return make_float2(x[u][k], x[u][k + 1]); };
#pragma unroll
        for (int u = 0; u < U; ++u) {
            float2 s = pair(u, 0);
#pragma unroll
            for (int k = 2; k < V; k += 2) s = add2(s, pair(u, k));
            sum[u] = s.x + s.y;
        }
        lanes_sum(sum, rt.lanes);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            sum[u] *= inv;
            float2 q = both(0.f);
#pragma unroll
            for (int k = 0; k < V; k += 2) {
                const float2 d = add2(pair(u, k), both(-sum[u]));
                q = fma2(d, d, q);
                x[u][k] = d.x;
                x[u][k + 1] = d.y;
            }
            sq[u] = on ? q.x + q.y : 0.f;   // the lanes that fill a group up hold no values
        }
        lanes_sum(sq, rt.lanes);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = base + u * step + slot;
            const float rstd = rsqrtf(fmaf(sq[u], inv, p.eps));
            if (on && row < p.N) {
#pragma unroll
                for (int k = 0; k < V; k += 2) {
                    const float2 y = act2<ACT>(fma2(mul2(pair(u, k), both(rstd)), make_float2(ch.gamma[k], ch.gamma[k + 1]),
                                                    make_float2(ch.beta[k], ch.beta[k + 1])));
                    x[u][k] = y.x;
                    x[u][k + 1] = y.y;
                }
                store_vec<E>(p.y, static_cast<size_t>(row) * p.C + c, pack(x[u], E{}));
                if ((threadIdx.x & (rt.lanes - 1)) == 0) {
                    const size_t g = static_cast<size_t>(row) * p.G + group;
                    if (p.mean) p.mean[g] = sum[u];
                    if (p.rstd) p.rstd[g] = rstd;
                }
            }
        }
    }
}

// Adds the threads' per-channel sums over the block's slots and writes them as
// partial `index`: part [.., 2, C], A (dbeta) then B (dgamma).
template <int V>
__device__ __forceinline__ void write_partial(const GnParams& p, float* smem, const float (&a)[V], const float (&b)[V],
                                              int slot, int slots, int tile, int c, int c0, bool on, long long index)
{
    float* out = p.part + static_cast<size_t>(index) * 2 * p.C;
    const int width = tile * V;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        __syncthreads();
        if (on)
#pragma unroll
            for (int k = 0; k < V; ++k) smem[slot * width + (c - c0) + k] = which ? b[k] : a[k];
        __syncthreads();
        for (int i = threadIdx.x; i < width && c0 + i < p.C; i += blockDim.x) {
            float s = 0.f;
            for (int k = 0; k < slots; ++k) s += smem[k * width + i];
            out[which * p.C + c0 + i] = s;
        }
    }
}

template <typename E, int ACT, int U>
__global__ void __launch_bounds__(kRowThreads, sizeof(E) == 4 ? 3 : 2) gn_rows_grad_kernel(const GnParams p)
{
    constexpr int V = vec<E>;
    __shared__ float s_part[kRowThreads * V];
    griddep_launch();
    const RowTile rt = row_tile<E>(p.C, p.G);
    const int slot = threadIdx.x / rt.tile, v = blockIdx.y * kRowThreads + threadIdx.x % rt.tile;
    const int group = v / rt.lanes, c = (group * rt.vecs + v % rt.lanes) * V;
    const int c0 = blockIdx.y * (kRowThreads / rt.lanes) * rt.vecs * V;   // the block's first channel
    const bool on = slot < rt.slots && group < p.G && v % rt.lanes < rt.vecs;
    const Channels<V> ch(p, on ? c : 0);
    const float inv = 1.f / static_cast<float>(rt.vecs * V);
    const long long step = static_cast<long long>(gridDim.x) * rt.slots;
    float A[V], B[V];
#pragma unroll
    for (int k = 0; k < V; ++k) A[k] = B[k] = 0.f;
    for (long long base = static_cast<long long>(blockIdx.x) * rt.slots; base < p.N; base += step * U) {
        uint4 rx[U], rd[U];
        float mean[U], rstd[U], s1[U], s2[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = base + u * step + slot;
            const bool ok = on && row < p.N;
            const size_t at = static_cast<size_t>(row) * p.C + c, g = static_cast<size_t>(row) * p.G + group;
            rx[u] = ok ? load_vec<E>(p.x, at) : make_uint4(0, 0, 0, 0);
            rd[u] = ok ? load_vec<E>(p.dy, at) : make_uint4(0, 0, 0, 0);
            mean[u] = ok ? __ldg(p.mean + g) : 0.f;
            rstd[u] = ok ? __ldg(p.rstd + g) : 0.f;
        }
        float x[U][V], d[U][V];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            unpack(rx[u], x[u], E{});
            unpack(rd[u], d[u], E{});
            s1[u] = s2[u] = 0.f;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float xh = (x[u][k] - mean[u]) * rstd[u];
                const float dz = d[u][k] * slope<ACT>(x[u][k], mean[u], rstd[u], ch.gamma[k], ch.beta[k], xh);
                A[k] += dz;
                B[k] = fmaf(dz, xh, B[k]);
                x[u][k] = xh;
                d[u][k] = dz * ch.gamma[k];
                s1[u] += d[u][k];
                s2[u] = fmaf(d[u][k], xh, s2[u]);
            }
        }
        lanes_sum(s1, rt.lanes);
        lanes_sum(s2, rt.lanes);
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const long long row = base + u * step + slot;
            const float m1 = s1[u] * inv, m2 = s2[u] * inv;
            if (on && row < p.N) {
#pragma unroll
                for (int k = 0; k < V; ++k) x[u][k] = rstd[u] * (d[u][k] - fmaf(x[u][k], m2, m1));
                store_vec<E>(p.dx, static_cast<size_t>(row) * p.C + c, pack(x[u], E{}));
            }
        }
    }
    if (p.dgamma || p.dbeta)
        write_partial<V>(p, s_part, A, B, slot, rt.slots, rt.tile / rt.lanes * rt.vecs, c, c0, on, blockIdx.x);
}

// dbeta, dgamma: the partials' sums over their index, in a fixed order.  Eight
// channels per block, so that every partial of a few hundred is in flight at once.
__global__ void __launch_bounds__(1024) gn_param_kernel(const GnParams p, long long partials)
{
    __shared__ float s[2][128][9];
    griddep_wait();
    const int t = threadIdx.x & 7, w = threadIdx.x >> 3, c = blockIdx.x * 8 + t;
    float a = 0.f, b = 0.f;
#pragma unroll 8
    for (long long i = w; i < partials; i += 128) {
        a += p.part[static_cast<size_t>(i) * 2 * p.C + c];
        b += p.part[static_cast<size_t>(i) * 2 * p.C + p.C + c];
    }
    s[0][w][t] = a;
    s[1][w][t] = b;
    for (int o = 64; o > 0; o >>= 1) {
        __syncthreads();
        if (w < o) {
            s[0][w][t] += s[0][w + o][t];
            s[1][w][t] += s[1][w + o][t];
        }
    }
    if (w == 0) {
        if (p.dbeta) p.dbeta[c] = s[0][0][t];
        if (p.dgamma) p.dgamma[c] = s[1][0][t];
    }
}

// ---------------------------------------------------------------- line
// One warp per (row, group) of any width; the row's values are read again from L1.
template <typename E, int ACT, bool GRAD>
__global__ void __launch_bounds__(128) gn_line_kernel(const GnParams p)
{
    const int lane = threadIdx.x & 31, width = p.C / p.G;
    const long long item = static_cast<long long>(blockIdx.x) * 4 + (threadIdx.x >> 5);
    if (item >= p.N * p.G) return;
    const int c0 = static_cast<int>(item % p.G) * width;
    const size_t at = static_cast<size_t>(item / p.G) * p.C + c0;
    const E* x = static_cast<const E*>(p.x) + at;
    const float inv = 1.f / static_cast<float>(width);
    auto gamma = [&](int i) { return p.gamma ? p.gamma[c0 + i] : 1.f; };
    auto beta = [&](int i) { return p.beta ? p.beta[c0 + i] : 0.f; };
    if constexpr (!GRAD) {
        float s = 0.f, q = 0.f;
        for (int i = lane; i < width; i += 32) s += to_f(x[i]);
        const float mean = warp_sum(s) * inv;
        for (int i = lane; i < width; i += 32) {
            const float d = to_f(x[i]) - mean;
            q = fmaf(d, d, q);
        }
        const float rstd = rsqrtf(fmaf(warp_sum(q), inv, p.eps));
        E* y = static_cast<E*>(p.y) + at;
        for (int i = lane; i < width; i += 32)
            y[i] = from_f<E>(act<ACT>(fmaf((to_f(x[i]) - mean) * rstd, gamma(i), beta(i))));
        if (lane == 0) {
            if (p.mean) p.mean[item] = mean;
            if (p.rstd) p.rstd[item] = rstd;
        }
    } else {
        const E* dy = static_cast<const E*>(p.dy) + at;
        const float mean = p.mean[item], rstd = p.rstd[item];
        float s1 = 0.f, s2 = 0.f;
        auto dh = [&](int i, float& xh) {
            const float xv = to_f(x[i]);
            xh = (xv - mean) * rstd;
            return to_f(dy[i]) * slope<ACT>(xv, mean, rstd, gamma(i), beta(i), xh) * gamma(i);
        };
        for (int i = lane; i < width; i += 32) {
            float xh;
            const float v = dh(i, xh);
            s1 += v;
            s2 = fmaf(v, xh, s2);
        }
        s1 = warp_sum(s1) * inv;
        s2 = warp_sum(s2) * inv;
        E* dx = static_cast<E*>(p.dx) + at;
        for (int i = lane; i < width; i += 32) {
            float xh;
            const float v = dh(i, xh);
            dx[i] = from_f<E>(rstd * (v - fmaf(xh, s2, s1)));
        }
    }
}

// ---------------------------------------------------------------- slab
struct SlabPlan {
    int threads, cluster;    // CTAs per cluster, each with `rows` positions
    int rows, groups, cblk;  // groups and channels of a channel block
    int grid_x;              // clusters * cluster
};

// Shared memory: the values (positions rounded up to whole passes of the
// slots), per-slot channel sums (two kinds in the backward pass) and its
// running sums, statistics of every group.
long long slab_smem(const SlabPlan& s, int e, bool grad)
{
    const int tile = s.cblk * e / 16, slots = s.threads / tile;
    const long long values = static_cast<long long>(s.rows + slots - 1) / slots * slots * tile * 16;
    return (grad ? 2 : 1) * (values + slots * s.cblk * 4) + (grad ? 2 * s.cblk * 4 : 0) + s.groups * 4 * 4;
}

template <typename E, int ACT, bool GRAD>
__global__ void __launch_bounds__(256) gn_slab_kernel(const GnParams p, const SlabPlan sp)
{
    constexpr int V = vec<E>;
    extern __shared__ __align__(128) unsigned char smem[];
    if constexpr (GRAD) griddep_launch();
    cg::cluster_group cluster = cg::this_cluster();
    const int rank = sp.cluster > 1 ? static_cast<int>(cluster.block_rank()) : 0;
    const int tile = sp.cblk / V, slots = sp.threads / tile, width = p.C / p.G;
    const int slot = threadIdx.x / tile, cl = threadIdx.x % tile * V, c0 = blockIdx.y * sp.cblk;
    const bool on = slot < slots;
    const long long r0 = static_cast<long long>(rank) * sp.rows;
    const int rows = static_cast<int>(max(0LL, min(static_cast<long long>(sp.rows), p.L - r0)));   // this CTA's positions
    const int mine = on && slot < rows ? (rows - slot + slots - 1) / slots : 0;                  // this thread's
    const int stride = slots * tile;   // vectors between a thread's consecutive positions
    const int per_cta = (sp.rows + slots - 1) / slots * stride;
    uint4* sx = reinterpret_cast<uint4*>(smem);
    uint4* sd = sx + per_cta;
    float* s_part = reinterpret_cast<float*>(sx + (GRAD ? 2 : 1) * per_cta);
    float* s_part2 = s_part + slots * sp.cblk;
    float* s_sum = s_part2 + (GRAD ? slots * sp.cblk : 0);    // backward: running A, B per channel
    float* s_stat = s_part + (GRAD ? 2 : 1) * slots * sp.cblk + (GRAD ? 2 * sp.cblk : 0);
    float* s_own = s_stat;                     // [groups][2]: this CTA's, read by the cluster
    float* s_all = s_stat + 2 * sp.groups;     // [groups][2]: the sample's
    const uint32_t ax = smem_u32(sx + threadIdx.x), ad = smem_u32(sd + threadIdx.x);
    const Channels<V> ch(p, c0 + cl);
    int gl[V];   // the local group of each channel
    gl[0] = cl / width;
    int left = width - cl % width;   // of that group, from channel k on
#pragma unroll
    for (int k = 1; k < V; ++k) {
        const bool next = --left == 0;
        gl[k] = gl[k - 1] + next;
        if (next) left = width;
    }
    const float count = static_cast<float>(rows) * width, total = static_cast<float>(p.L) * width;
    if constexpr (GRAD)
        for (int i = threadIdx.x; i < 2 * sp.cblk; i += sp.threads) s_sum[i] = 0.f;

    // Per-slot sums of units, a thread's vector where groups are whole vectors and else a channel; a group's
    // `per` units over all slots together.
    const bool whole = width % V == 0;
    const int units = whole ? tile : sp.cblk, per = whole ? width / V : width;
    auto put = [&](const float (&v)[V]) {
        if (!on) return;
        if (whole) {
            float s = 0.f;
#pragma unroll
            for (int k = 0; k < V; ++k) s += v[k];
            s_part[slot * units + cl / V] = s;
        } else {
#pragma unroll
            for (int k = 0; k < V; ++k) s_part[slot * units + cl + k] = v[k];
        }
    };
    // Sums of each group, by `sub` neighbouring lanes: as many as make the groups fill the block (a warp for each
    // of 32 groups in turn took 22.6 us for 29 samples of 3 x 96).
    int sub = 32;
    while (sub > 1 && sp.groups * sub > sp.threads) sub >>= 1;
    const int sl = threadIdx.x & (sub - 1);
    auto each_group = [&](auto&& terms, auto&& done) {
        for (int g0 = 0; g0 < sp.groups; g0 += sp.threads / sub) {
            const int g = g0 + static_cast<int>(threadIdx.x) / sub;
            float v[2] = {0.f, 0.f};
            if (g < sp.groups) terms(g, v);
            lanes_sum(v, sub);
            if (sl == 0 && g < sp.groups) done(g, v);
        }
    };
    auto slots_of = [&](int g, float (&v)[2]) {   // the group's units over all slots
        if ((per & (per - 1)) == 0 && per <= sub) {
            for (int i = sl / per; i < slots; i += sub / per) v[0] += s_part[i * units + g * per + (sl & (per - 1))];
        } else {
            for (int i = sl; i < slots * per; i += sub) v[0] += s_part[i / per * units + g * per + i % per];
        }
    };

    const long long clusters = gridDim.x / sp.cluster;
    for (long long n = blockIdx.x / sp.cluster; n < p.N; n += clusters) {
        const size_t at0 = (static_cast<size_t>(n) * p.L + r0 + slot) * p.C + c0 + cl;
        for (int i = 0; i < mine; ++i) {
            const size_t at = at0 + static_cast<size_t>(i) * slots * p.C;
            cp_async16(ax + i * stride * 16, static_cast<const E*>(p.x) + at, true);
            if constexpr (GRAD) cp_async16(ad + i * stride * 16, static_cast<const E*>(p.dy) + at, true);
        }
        cp_async_commit();
        float mean[V], rstd[V];
        if constexpr (GRAD) {
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const size_t g = static_cast<size_t>(n) * p.G + c0 / width + gl[k];
                mean[k] = p.mean[g];
                rstd[k] = p.rstd[g];
            }
        }
        cp_async_wait<0>();   // a thread reads only what it copied
        float a[V], b[V];
#pragma unroll
        for (int k = 0; k < V; ++k) a[k] = b[k] = 0.f;
        if constexpr (!GRAD) {
            for (int i = 0; i < mine; ++i) {
                float x[V];
                unpack(sx[threadIdx.x + i * stride], x, E{});
#pragma unroll
                for (int k = 0; k < V; ++k) a[k] += x[k];
            }
            put(a);
            __syncthreads();
            each_group(slots_of, [&](int g, const float (&v)[2]) { s_own[2 * g] = rows > 0 ? v[0] / count : 0.f; });
            __syncthreads();
#pragma unroll
            for (int k = 0; k < V; ++k) mean[k] = s_own[2 * gl[k]];
            for (int i = 0; i < mine; ++i) {
                float x[V];
                unpack(sx[threadIdx.x + i * stride], x, E{});
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float d = x[k] - mean[k];
                    b[k] = fmaf(d, d, b[k]);
                }
            }
            put(b);
            __syncthreads();
            each_group(slots_of, [&](int g, const float (&v)[2]) { s_own[2 * g + 1] = v[0]; });
            if (sp.cluster > 1) cluster.sync(); else __syncthreads();
            for (int g = threadIdx.x; g < sp.groups; g += sp.threads) {
                Stat s{0.f, 0.f, 0.f};
                for (int r = 0; r < sp.cluster; ++r) {
                    const float* o = sp.cluster > 1 ? cluster.map_shared_rank(s_own, r) : s_own;
                    const float rr = static_cast<float>(max(0LL, min(static_cast<long long>(sp.rows), p.L - static_cast<long long>(r) * sp.rows)));
                    s = merge(s, Stat{rr * width, o[2 * g], o[2 * g + 1]});
                }
                const float rs = rsqrtf(s.m2 / total + p.eps);
                s_all[2 * g] = s.mean;
                s_all[2 * g + 1] = rs;
                if (rank == 0) {
                    const size_t gi = static_cast<size_t>(n) * p.G + c0 / width + g;
                    if (p.mean) p.mean[gi] = s.mean;
                    if (p.rstd) p.rstd[gi] = rs;
                }
            }
            __syncthreads();
#pragma unroll
            for (int k = 0; k < V; ++k) {
                mean[k] = s_all[2 * gl[k]];
                rstd[k] = s_all[2 * gl[k] + 1] * ch.gamma[k];
            }
            for (int i = 0; i < mine; ++i) {
                float x[V];
                unpack(sx[threadIdx.x + i * stride], x, E{});
#pragma unroll
                for (int k = 0; k < V; k += 2) {
                    const float2 d = add2(make_float2(x[k], x[k + 1]), make_float2(-mean[k], -mean[k + 1]));
                    const float2 y = act2<ACT>(fma2(d, make_float2(rstd[k], rstd[k + 1]), make_float2(ch.beta[k], ch.beta[k + 1])));
                    x[k] = y.x;
                    x[k + 1] = y.y;
                }
                store_vec<E>(p.y, at0 + static_cast<size_t>(i) * slots * p.C, pack(x, E{}));
            }
        } else {
            for (int i = 0; i < mine; ++i) {
                float x[V], d[V];
                unpack(sx[threadIdx.x + i * stride], x, E{});
                unpack(sd[threadIdx.x + i * stride], d, E{});
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float xh = (x[k] - mean[k]) * rstd[k];
                    const float dz = d[k] * slope<ACT>(x[k], mean[k], rstd[k], ch.gamma[k], ch.beta[k], xh);
                    a[k] += dz;
                    b[k] = fmaf(dz, xh, b[k]);
                    d[k] = dz;
                }
                // dy or 0: kept, so that the second pass does not ask for the slope again
                if constexpr (ACT == SRWM_ACT_RELU) sd[threadIdx.x + i * stride] = pack(d, E{});
            }
            if (on)
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    s_part[slot * sp.cblk + cl + k] = a[k];
                    s_part2[slot * sp.cblk + cl + k] = b[k];
                }
            __syncthreads();
            for (int c = threadIdx.x; c < sp.cblk; c += sp.threads) {   // slots together; into the running sums
                float sa = 0.f, sb = 0.f;
                for (int i = 0; i < slots; ++i) {
                    sa += s_part[i * sp.cblk + c];
                    sb += s_part2[i * sp.cblk + c];
                }
                s_sum[c] += sa;
                s_sum[sp.cblk + c] += sb;
                s_part[c] = sa;      // only this thread reads or writes column c from here to the barrier
                s_part2[c] = sb;
            }
            __syncthreads();
            each_group(
                [&](int g, float (&v)[2]) {
                    for (int i = sl; i < width; i += sub) {
                        const float ga = p.gamma ? p.gamma[c0 + g * width + i] : 1.f;
                        v[0] = fmaf(ga, s_part[g * width + i], v[0]);
                        v[1] = fmaf(ga, s_part2[g * width + i], v[1]);
                    }
                },
                [&](int g, const float (&v)[2]) {
                    s_own[2 * g] = v[0];
                    s_own[2 * g + 1] = v[1];
                });
            if (sp.cluster > 1) cluster.sync(); else __syncthreads();
            for (int g = threadIdx.x; g < sp.groups; g += sp.threads) {
                float u = 0.f, w = 0.f;
                for (int r = 0; r < sp.cluster; ++r) {
                    const float* o = sp.cluster > 1 ? cluster.map_shared_rank(s_own, r) : s_own;
                    u += o[2 * g];
                    w += o[2 * g + 1];
                }
                s_all[2 * g] = u / total;
                s_all[2 * g + 1] = w / total;
            }
            __syncthreads();
            float m1[V], m2[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                m1[k] = s_all[2 * gl[k]];
                m2[k] = s_all[2 * gl[k] + 1];
            }
            for (int i = 0; i < mine; ++i) {
                float x[V], d[V];
                unpack(sx[threadIdx.x + i * stride], x, E{});
                unpack(sd[threadIdx.x + i * stride], d, E{});
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float xh = (x[k] - mean[k]) * rstd[k];
                    float dz = d[k];
                    if constexpr (ACT != SRWM_ACT_RELU)
                        dz *= slope<ACT>(x[k], mean[k], rstd[k], ch.gamma[k], ch.beta[k], xh);
                    x[k] = rstd[k] * (dz * ch.gamma[k] - fmaf(xh, m2[k], m1[k]));
                }
                store_vec<E>(p.dx, at0 + static_cast<size_t>(i) * slots * p.C, pack(x, E{}));
            }
        }
        // the cluster has read this CTA's statistics before they change or it exits
        if (sp.cluster > 1) cluster.sync(); else __syncthreads();
    }
    if constexpr (GRAD) {
        if (p.dgamma || p.dbeta) {
            float* out = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.C + c0;
            for (int c = threadIdx.x; c < sp.cblk; c += sp.threads) {
                out[c] = s_sum[c];
                out[p.C + c] = s_sum[sp.cblk + c];
            }
        }
    }
}

// ---------------------------------------------------------------- split
// Scratch: per sample, range of positions and channel (mean, M2) or (A, B) as
// [N][ranges][2][C]; then per sample and group (mean, rstd) or (m1, m2).
struct SplitPlan {
    int rows, ranges;   // positions of a range
};

__device__ __forceinline__ float* split_groups(const GnParams& p, const SplitPlan& s)
{
    return p.part + static_cast<size_t>(p.N) * s.ranges * 2 * p.C;
}

// STAGE 0: a range's per-channel values; 1: the second pass over it.
template <typename E, int ACT, bool GRAD, int STAGE>
__global__ void __launch_bounds__(kRowThreads) gn_split_kernel(const GnParams p, const SplitPlan sp)
{
    constexpr int V = vec<E>;
    __shared__ float s_part[kRowThreads * V];
    griddep_launch();
    if constexpr (STAGE == 1) griddep_wait();
    const int cv = p.C / V, tile = min(cv, kRowThreads), slots = kRowThreads / tile, width = p.C / p.G;
    const int slot = threadIdx.x / tile, c0 = blockIdx.y * kRowThreads * V, c = c0 + threadIdx.x % tile * V;
    const bool on = slot < slots && c < p.C;
    const long long n = blockIdx.x / sp.ranges, range = blockIdx.x % sp.ranges;
    const long long r0 = range * sp.rows, r1 = min(r0 + sp.rows, p.L);
    const Channels<V> ch(p, on ? c : 0);
    float mean[V], rstd[V], m1[V], m2[V];
    if (GRAD || STAGE == 1)
#pragma unroll
        for (int k = 0; k < V; ++k) {
            const size_t g = static_cast<size_t>(n) * p.G + (on ? c + k : 0) / width;
            const float* st = split_groups(p, sp) + 2 * g;
            mean[k] = GRAD ? p.mean[g] : st[0];
            rstd[k] = GRAD ? p.rstd[g] : st[1];
            m1[k] = GRAD && STAGE == 1 ? st[0] : 0.f;
            m2[k] = GRAD && STAGE == 1 ? st[1] : 0.f;
        }
    float a[V], b[V], seen = 0.f;
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] = b[k] = 0.f;
    if (on)
#pragma unroll 4
        for (long long r = r0 + slot; r < r1; r += slots) {
            const size_t at = (static_cast<size_t>(n) * p.L + r) * p.C + c;
            float x[V], d[V];
            unpack(load_vec<E>(p.x, at), x, E{});
            if constexpr (GRAD) unpack(load_vec<E>(p.dy, at), d, E{});
            if constexpr (!GRAD && STAGE == 0) {
                seen += 1.f;
                const float f = __fdividef(1.f, seen);
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float e = x[k] - a[k];
                    a[k] = fmaf(e, f, a[k]);
                    b[k] = fmaf(e, x[k] - a[k], b[k]);
                }
            } else if constexpr (!GRAD) {
#pragma unroll
                for (int k = 0; k < V; ++k) x[k] = act<ACT>(fmaf((x[k] - mean[k]) * rstd[k], ch.gamma[k], ch.beta[k]));
                store_vec<E>(p.y, at, pack(x, E{}));
            } else {
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float xh = (x[k] - mean[k]) * rstd[k];
                    const float dz = d[k] * slope<ACT>(x[k], mean[k], rstd[k], ch.gamma[k], ch.beta[k], xh);
                    if constexpr (STAGE == 0) {
                        a[k] += dz;
                        b[k] = fmaf(dz, xh, b[k]);
                    } else {
                        x[k] = rstd[k] * (dz * ch.gamma[k] - fmaf(xh, m2[k], m1[k]));
                    }
                }
                if constexpr (STAGE == 1) store_vec<E>(p.dx, at, pack(x, E{}));
            }
        }
    if constexpr (STAGE == 1) return;
    if constexpr (GRAD) {
        write_partial<V>(p, s_part, a, b, slot, slots, tile, c, c0, on, blockIdx.x);
    } else {
        // the slots' statistics of a channel together: means first, then M2 beside the merged mean
        __shared__ float s_part2[kRowThreads * V];
        const int wide = tile * V;
        if (on)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                s_part[slot * wide + (c - c0) + k] = a[k];
                s_part2[slot * wide + (c - c0) + k] = b[k];
            }
        __syncthreads();
        float* out = p.part + static_cast<size_t>(blockIdx.x) * 2 * p.C;
        for (int i = threadIdx.x; i < wide && c0 + i < p.C; i += kRowThreads) {
            Stat s{0.f, 0.f, 0.f};
            for (int k = 0; k < slots; ++k) {
                const long long rows = r1 - r0 > k ? (r1 - r0 - k + slots - 1) / slots : 0;
                s = merge(s, Stat{static_cast<float>(rows), s_part[k * wide + i], s_part2[k * wide + i]});
            }
            out[c0 + i] = s.mean;
            out[p.C + c0 + i] = s.m2;
        }
    }
}

// One CTA per sample and group: its ranges' and channels' values together.  A
// thread keeps one channel (or steps over channels where the group is wider
// than the block), so that its loads of several ranges are in flight at once.
constexpr int kMergeThreads = 1024;

template <bool GRAD>
__global__ void __launch_bounds__(kMergeThreads) gn_merge_kernel(const GnParams p, const SplitPlan sp)
{
    __shared__ float s0[kMergeThreads], s1[kMergeThreads], s2[kMergeThreads];
    griddep_launch();
    griddep_wait();
    const long long n = blockIdx.x / p.G;
    const int g = blockIdx.x % p.G, width = p.C / p.G, t = threadIdx.x;
    const int across = min(width, kMergeThreads), deep = kMergeThreads / across;   // channels, ranges at a time
    const float* in = p.part + static_cast<size_t>(n) * sp.ranges * 2 * p.C + g * width;
    Stat s{0.f, 0.f, 0.f};
    if (t < across * deep)
        for (int c = t % across; c < width; c += across) {
            const float ga = GRAD && p.gamma ? p.gamma[g * width + c] : 1.f;
#pragma unroll 4
            for (int range = t / across; range < sp.ranges; range += deep) {
                const float* at = in + static_cast<size_t>(range) * 2 * p.C + c;
                const float u = at[0], w = at[p.C];
                if constexpr (GRAD) {
                    s.mean = fmaf(ga, u, s.mean);
                    s.m2 = fmaf(ga, w, s.m2);
                } else {
                    const long long rows = min(static_cast<long long>(sp.rows), p.L - static_cast<long long>(range) * sp.rows);
                    s = merge(s, Stat{static_cast<float>(rows), u, w});
                }
            }
        }
    s0[t] = s.n, s1[t] = s.mean, s2[t] = s.m2;
    for (int o = kMergeThreads / 2; o > 0; o >>= 1) {
        __syncthreads();
        if (t < o) {
            if constexpr (GRAD) {
                s1[t] += s1[t + o];
                s2[t] += s2[t + o];
            } else {
                const Stat m = merge(Stat{s0[t], s1[t], s2[t]}, Stat{s0[t + o], s1[t + o], s2[t + o]});
                s0[t] = m.n, s1[t] = m.mean, s2[t] = m.m2;
            }
        }
    }
    if (t == 0) {
        const float total = static_cast<float>(p.L) * width;
        float* out = split_groups(p, sp) + 2 * static_cast<size_t>(blockIdx.x);
        if constexpr (GRAD) {
            out[0] = s1[0] / total;
            out[1] = s2[0] / total;
        } else {
            const float rstd = rsqrtf(s2[0] / total + p.eps);
            out[0] = s1[0];
            out[1] = rstd;
            if (p.mean) p.mean[blockIdx.x] = s1[0];
            if (p.rstd) p.rstd[blockIdx.x] = rstd;
        }
    }
}

// dz's channel sums over ranges of rows with statistics of their own (L = 1, the line way).
template <typename E, int ACT>
__global__ void __launch_bounds__(kRowThreads) gn_line_param_kernel(const GnParams p, long long rows)
{
    constexpr int V = vec<E>;
    __shared__ float s_part[kRowThreads * V];
    griddep_launch();
    const int tile = min(p.C / V, kRowThreads), slots = kRowThreads / tile, width = p.C / p.G;
    const int slot = threadIdx.x / tile, c0 = blockIdx.y * kRowThreads * V, c = c0 + threadIdx.x % tile * V;
    const bool on = slot < slots && c < p.C;
    const Channels<V> ch(p, on ? c : 0);
    float a[V], b[V];
#pragma unroll
    for (int k = 0; k < V; ++k) a[k] = b[k] = 0.f;
    const long long r0 = blockIdx.x * rows, r1 = min(r0 + rows, p.N);
    if (on)
        for (long long r = r0 + slot; r < r1; r += slots) {
            float x[V], d[V];
            unpack(load_vec<E>(p.x, static_cast<size_t>(r) * p.C + c), x, E{});
            unpack(load_vec<E>(p.dy, static_cast<size_t>(r) * p.C + c), d, E{});
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const size_t g = static_cast<size_t>(r) * p.G + (c + k) / width;
                const float mean = p.mean[g], rstd = p.rstd[g], xh = (x[k] - mean) * rstd;
                const float dz = d[k] * slope<ACT>(x[k], mean, rstd, ch.gamma[k], ch.beta[k], xh);
                a[k] += dz;
                b[k] = fmaf(dz, xh, b[k]);
            }
        }
    write_partial<V>(p, s_part, a, b, slot, slots, tile, c, c0, on, blockIdx.x);
}

// ---------------------------------------------------------------- the choice
enum Way { kRows, kLine, kSlab, kSplit };

struct GnPlan {
    Way way;
    SlabPlan slab;
    SplitPlan split;
    int grid_x, grid_y;
    long long partials;   // of the parameter gradients
    size_t scratch;       // floats
};

GnPlan gn_plan(int e, long long N, long long L, int C, int G, bool grad)
{
    GnPlan g{};
    const int V = 16 / e, cv = C / V, width = C / G;
    g.grid_y = (cv + kRowThreads - 1) / kRowThreads;
    if (L == 1 && width % V == 0 && width / V <= 32) {
        g.way = kRows;
        const RowTile rt = e == 4 ? row_tile<float>(C, G) : row_tile<__half>(C, G);
        const int slots = rt.slots;
        g.grid_y = (G * rt.lanes + kRowThreads - 1) / kRowThreads;
        const long long blocks = (N + slots - 1) / slots;
        // what the GPU holds at once: a block keeps its channels' gamma, beta and sums over its rows
        g.grid_x = static_cast<int>(std::max(1LL, std::min(blocks, static_cast<long long>(kSms) * (grad && e == 2 ? 2 : 3))));
        g.partials = g.grid_x;
        g.scratch = grad ? static_cast<size_t>(g.partials) * 2 * C : 0;
        return g;
    }
    if (L == 1) {
        g.way = kLine;
        g.grid_x = static_cast<int>((N * G + 3) / 4);
        g.partials = std::max(1LL, std::min((N + 31) / 32, 4LL * kSms));
        g.scratch = grad ? static_cast<size_t>(g.partials) * 2 * C : 0;
        return g;
    }
    // The slab: as few CTAs per sample as hold it well; more of them, or fewer
    // channels each, while a CTA holds too much or the GPU is not filled.  Large
    // inputs are split by channels down to 256 bytes of a position, then by
    // positions, then by channels down to 64 bytes, small ones by channels first
    // (101 x 441 x 64 in bf16 backward: 13.3 us by positions, 11.7 by channels;
    // 208 x 1764 x 64 in fp32 forward: 44 and 68): a cluster's exchange costs a
    // small call more than short pieces of memory do.  48 MB lie between the two;
    // more positions move the border down (700 x 441 x 64 in bf16 forward, 38 MB:
    // 28.0 by positions, 25.3 by channels; 110 x 1764 x 64 in bf16, 24 MB: 20.0 and
    // 22.2, in fp32, 47 MB: 24.3 and 31.4), which the rule does not follow.
    SlabPlan s{};
    s.cluster = 1;
    s.groups = G;
    const long long copies = grad ? 2 : 1;
    const bool small = copies * N * L * C * e < (48 << 20);
    auto bytes = [&] { return copies * ((L + s.cluster - 1) / s.cluster) * s.groups * width * e; };
    auto can_halve = [&](int least) {   // to pieces of at least so many bytes of a position
        return s.groups % 2 == 0 && (s.groups / 2 * width) % V == 0 && s.groups / 2 * width * e >= least;
    };
    while (s.groups * width / V > 256 && s.groups % 2 == 0 && (s.groups / 2 * width) % V == 0) s.groups /= 2;
    for (;;) {
        const bool full = N * s.cluster * (G / s.groups) >= 2 * kSms;
        if (bytes() <= kSlabGood && (full || bytes() <= 8192)) break;
        if (can_halve(small ? 32 : 256))
            s.groups /= 2;
        else if (s.cluster < kMaxCluster && L >= 2 * s.cluster)
            s.cluster *= 2;
        else if (can_halve(64))
            s.groups /= 2;
        else
            break;
    }
    s.cblk = s.groups * width;
    const int tile = s.cblk / V;
    s.rows = static_cast<int>((L + s.cluster - 1) / s.cluster);
    const long long vectors = static_cast<long long>(s.rows) * tile;
    // fewer threads per sum to exchange; more where one or two CTAs have an SM to themselves (gradients in bf16 with 256 and
    // 128 threads: 300 x 7000 x 64 517 and 586 us, 600 x 1200 x 64 154 and 110)
    s.threads = bytes() > 80 * 1024 ? 256 : vectors >= 512 ? 128 : vectors >= 128 ? 64 : 32;
    while (s.threads < tile) s.threads *= 2;
    // fp32 gradients leave room for a second CTA on the SM, or the split way is faster though it reads x and dy twice
    // (76 x 1718 x 256: 175 us with one CTA, 122 split; 64 x 3136 x 64: 66 and 58).  In bf16 the slab keeps its lead
    // (32 x 9447 x 64: 87 and 102), and so does the forward pass (1 x 8000 x 512 in bf16: 13 and 28).
    if (tile <= 256 && slab_smem(s, e, grad) <= (grad && e == 4 ? kSmemPair : kSmemMost)) {
        g.way = kSlab;
        g.grid_y = G / s.groups;
        // the backward pass keeps its channel sums over several samples: fewer partials
        const long long clusters = grad ? std::max(1LL, std::min(N, static_cast<long long>(kSms) * 8 / s.cluster)) : N;
        g.grid_x = static_cast<int>(std::min(clusters, 0x7fffffffLL / s.cluster) * s.cluster);
        s.grid_x = g.grid_x;
        g.slab = s;
        g.partials = g.grid_x;
        g.scratch = grad ? static_cast<size_t>(g.partials) * 2 * C : 0;
        return g;
    }
    g.way = kSplit;
    const long long want = std::max(1LL, 8LL * kSms / std::max(1LL, N * g.grid_y));   // ranges to fill the GPU
    long long ranges = std::min(want, (L + 15) / 16);
    g.split.rows = static_cast<int>((L + ranges - 1) / ranges);
    g.split.ranges = static_cast<int>((L + g.split.rows - 1) / g.split.rows);
    g.grid_x = static_cast<int>(N * g.split.ranges);
    g.partials = N * g.split.ranges;
    g.scratch = static_cast<size_t>(g.partials) * 2 * C + static_cast<size_t>(N) * G * 2;
    return g;
}

int allow_smem(const void* kernel, std::atomic<bool>* done)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    if (done[dev].load()) return SRWM_OK;
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemMost) != cudaSuccess) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    done[dev].store(true);
    return SRWM_OK;
}

template <typename E, int ACT, bool GRAD>
int launch_slab(const GnParams& p, const GnPlan& g, cudaStream_t st)
{
    static std::atomic<bool> ok[kMaxDevices];
    auto kernel = gn_slab_kernel<E, ACT, GRAD>;
    const int rc = allow_smem(reinterpret_cast<const void*>(kernel), ok);
    if (rc != SRWM_OK) return rc;
    const SlabPlan& s = g.slab;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3(g.grid_x, g.grid_y);
    cfg.blockDim = dim3(s.threads);
    cfg.dynamicSmemBytes = static_cast<size_t>(slab_smem(s, sizeof(E), GRAD));
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeClusterDimension;
    attr.val.clusterDim.x = s.cluster;
    attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, p, s) != cudaSuccess) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    return SRWM_OK;
}

template <typename E, int ACT>
int forward(const GnParams& p, cudaStream_t st)
{
    const GnPlan g = gn_plan(sizeof(E), p.N, p.L, p.C, p.G, false);
    if (g.way == kRows)
        gn_rows_kernel<E, ACT, 4><<<dim3(g.grid_x, g.grid_y), kRowThreads, 0, st>>>(p);
    else if (g.way == kLine)
        gn_line_kernel<E, ACT, false><<<g.grid_x, 128, 0, st>>>(p);
    else if (g.way == kSlab)
        return launch_slab<E, ACT, false>(p, g, st);
    else {
        const dim3 grid(g.grid_x, g.grid_y);
        gn_split_kernel<E, ACT, false, 0><<<grid, kRowThreads, 0, st>>>(p, g.split);
        int rc = launched();
        if (rc == SRWM_OK)
            rc = launch_behind(gn_merge_kernel<false>, dim3(static_cast<unsigned>(p.N * p.G)), kMergeThreads, 0, st, p, g.split);
        return rc == SRWM_OK ? launch_behind(gn_split_kernel<E, ACT, false, 1>, grid, kRowThreads, 0, st, p, g.split) : rc;
    }
    return launched();
}

template <typename E, int ACT>
int backward(const GnParams& p, cudaStream_t st)
{
    GnPlan g = gn_plan(sizeof(E), p.N, p.L, p.C, p.G, true);
    const bool params = p.dgamma || p.dbeta;
    int rc = SRWM_OK;
    if (p.N == 0)
        g.partials = 0;
    else if (g.way == kRows)
        gn_rows_grad_kernel<E, ACT, 16 / vec<E>><<<dim3(g.grid_x, g.grid_y), kRowThreads, 0, st>>>(p);
    else if (g.way == kLine) {
        gn_line_kernel<E, ACT, true><<<g.grid_x, 128, 0, st>>>(p);
        if (params)
            gn_line_param_kernel<E, ACT><<<dim3(static_cast<unsigned>(g.partials), g.grid_y), kRowThreads, 0, st>>>(
                p, (p.N + g.partials - 1) / g.partials);
    } else if (g.way == kSlab)
        rc = launch_slab<E, ACT, true>(p, g, st);
    else {
        const dim3 grid(g.grid_x, g.grid_y);
        gn_split_kernel<E, ACT, true, 0><<<grid, kRowThreads, 0, st>>>(p, g.split);
        rc = launched();
        if (rc == SRWM_OK)
            rc = launch_behind(gn_merge_kernel<true>, dim3(static_cast<unsigned>(p.N * p.G)), kMergeThreads, 0, st, p, g.split);
        if (rc == SRWM_OK) rc = launch_behind(gn_split_kernel<E, ACT, true, 1>, grid, kRowThreads, 0, st, p, g.split);
    }
    if (rc == SRWM_OK) rc = launched();
    if (rc != SRWM_OK) return rc;
    return params ? launch_behind(gn_param_kernel, dim3(p.C / 8), 1024, 0, st, p, g.partials) : SRWM_OK;
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

// Enough for either width of type: the call's own plan may need less.
size_t scratch(long long N, long long L, int C, int G, bool grad)
{
    const size_t a = gn_plan(4, N, L, C, G, grad).scratch, b = gn_plan(2, N, L, C, G, grad).scratch;
    return std::max<size_t>(256, round256(std::max(a, b) * 4));
}

}  // namespace

size_t groupnorm_scratch(long long N, long long L, int C, int G) { return scratch(N, L, C, G, false); }
size_t groupnorm_backward_scratch(long long N, long long L, int C, int G) { return scratch(N, L, C, G, true); }

int groupnorm_launch(int dtype, int activation, const GnParams& p, cudaStream_t st)
{
    return p.N == 0 ? SRWM_OK : by_type(false, dtype, activation, p, st);
}

int groupnorm_backward_launch(int dtype, int activation, const GnParams& p, cudaStream_t st)
{
    return by_type(true, dtype, activation, p, st);
}

}  // namespace srwm
