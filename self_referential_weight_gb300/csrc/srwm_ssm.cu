// srwm_ssm.cu -- the selective state space scan: prompts and single tokens.
//
//   s_t = softplus(dt_t + dt_bias),  h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,
//   y_t = (C_t . h_t + skip u_t) silu(z_t)
// per channel, with N states each.  A CTA takes a range of channels of one
// sequence (or of a segment of it) in tiles of TT tokens: u, dt, z, B and C come
// by asynchronous copies a tile ahead; each warp forms its channels' steps and
// inputs in fp32, runs its states (in registers throughout) over the tile, and
// gates and stores the outputs.  Past a sequence's end a token's step is 0, which
// leaves the state as it is.
// Few streams: the axis is cut into segments.  A first kernel runs every segment
// but the last from a zero state; the second starts each from the states before
// it, H = exp(A sum s) H + H', and writes y.
#include <cuda_runtime.h>

#include <algorithm>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_ssm.cuh"

namespace srwm {
namespace {

using namespace ssm;

constexpr int TT = 16;   // tokens of a tile
constexpr int kSms = 152;

template <typename E, int N>
struct Tile {
    using L = Lay<N>;
    static constexpr int kCh = L::kCh;
    static constexpr int kRow = kCh * static_cast<int>(sizeof(E));            // bytes of a token's channels
    static constexpr int kBc = N * static_cast<int>(sizeof(E));               // and of its B (or C)
    static constexpr int kStage = TT * (3 * kRow + 2 * kBc);                  // u | dt | z | B | C as they land
    static constexpr int kWide = TT * (2 * kCh + 2 * N) * 4;                  // steps | inputs (then outputs) | B | C in fp32
    static constexpr int kSmem = 2 * kStage + kWide + 2 * kCh * 4;            // and dt_bias | skip
};

template <typename E, int N, bool OUT>
__global__ void __launch_bounds__(kThreads) ssm_kernel(const __grid_constant__ SsmParams p)
{
    using S = Tile<E, N>;
    using L = Lay<N>;
    constexpr int V = vec<E>, CH = S::kCh, WCH = L::kWarpCh;
    constexpr int PIECES = TT * WCH / V;   // of a warp's tile
    extern __shared__ __align__(128) unsigned char smem[];
    float* const steps = reinterpret_cast<float*>(smem + 2 * S::kStage);
    float* const xs = steps + TT * CH;
    float* const Bf = xs + TT * CH;
    float* const Cf = Bf + TT * N;
    float* const bias = Cf + TT * N;
    float* const skip = bias + CH;

    const Place w = place_of<CH>(p);
    const int n = valid_tokens(p.lengths, w.b, p.T);
    const int t0 = w.segment * p.seg_len, t1 = min(p.T, t0 + p.seg_len), live = min(n, t1);
    const int last = n > 0 ? (n - 1) / p.seg_len : 0;   // the segment at whose end the sequence ends
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp * WCH + lane / L::kLanes * 4, n4 = lane % L::kLanes * 4;   // this lane's channels and states
    const bool on = quad < w.count;
    if (!OUT && w.segment >= last) return;   // nothing comes after it

    E* const y = static_cast<E*>(p.y) + static_cast<size_t>(w.b) * p.T * p.D + w.first;
    if constexpr (OUT)   // rows past the end
        for (int i = threadIdx.x; i < (t1 - max(t0, live)) * (w.count / V); i += kThreads)
            store_vec<E>(y, static_cast<size_t>(max(t0, live) + i / (w.count / V)) * p.D + i % (w.count / V) * V, make_uint4(0, 0, 0, 0));
    if (w.segment > last) return;

    for (int i = threadIdx.x; i < CH; i += kThreads) {
        bias[i] = i < w.count && p.dt_bias ? p.dt_bias[w.first + i] : 0.f;
        skip[i] = i < w.count && p.skip ? p.skip[w.first + i] : 0.f;
    }
    const size_t tokens = static_cast<size_t>(w.b) * p.T;
    const E* const rows[3] = {static_cast<const E*>(p.u) + tokens * p.ld_u + w.first,
                              static_cast<const E*>(p.dt) + tokens * p.ld_dt + w.first,
                              static_cast<const E*>(p.z) + (p.z ? tokens * p.ld_z + w.first : 0)};
    const long long lds[3] = {p.ld_u, p.ld_dt, p.ld_z};
    const E* const bc[2] = {static_cast<const E*>(p.Bt) + tokens * p.ld_bc + w.group * N,
                            static_cast<const E*>(p.Ct) + tokens * p.ld_bc + w.group * N};
    const bool gated = OUT && p.z;
    auto load = [&](int tile) {
        const uint32_t to = smem_u32(smem) + (tile & 1) * S::kStage;
        const int first = t0 + tile * TT;
#pragma unroll
        for (int k = 0; k < 3; ++k) {
            if (k == 2 && !gated) continue;
#pragma unroll
            for (int i = 0; i < PIECES; i += 32) {   // a warp's own channels
                const int piece = i + lane, r = piece / (WCH / V), c = warp * WCH + piece % (WCH / V) * V;
                const bool ok = piece < PIECES && first + r < live && c < w.count;
                if (piece < PIECES)
                    cp_async16(to + k * TT * S::kRow + r * S::kRow + c * static_cast<int>(sizeof(E)),
                               rows[k] + (ok ? static_cast<long long>(first + r) * lds[k] + c : 0), ok);
            }
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            if (k == 1 && !OUT) continue;
            for (int i = threadIdx.x; i < TT * N / V; i += kThreads) {
                const int r = i / (N / V), c = i % (N / V) * V;
                const bool ok = first + r < live;
                cp_async16(to + 3 * TT * S::kRow + (k * TT + r) * S::kBc + c * static_cast<int>(sizeof(E)),
                           bc[k] + (ok ? static_cast<long long>(first + r) * p.ld_bc + c : 0), ok);
            }
        }
    };
    const int tiles = live > t0 ? (live - t0 + TT - 1) / TT : 0;
    if (tiles > 0) load(0);
    cp_async_commit();

    const size_t mat = (static_cast<size_t>(w.b) * p.D + w.first + quad) * N + n4, all = static_cast<size_t>(p.B) * p.D * N;
    float2 A[2][4], h[2][4];
    load_states(p.A + static_cast<size_t>(w.first + quad) * N + n4, N, on, A);
    load_states(p.h_in + mat, N, OUT && on && p.h_in, h);
    if (OUT && w.segment > 0) {
        griddep_wait();
        for (int j = 0; j < w.segment; ++j) {
            float2 own[2][4];
            load_states(p.seg_state + j * all + mat, N, on, own);
            const float4 d = on ? *reinterpret_cast<const float4*>(p.seg_dt + (static_cast<size_t>(j) * p.B + w.b) * p.D + w.first + quad)
                                : make_float4(0.f, 0.f, 0.f, 0.f);
            const float2 sum[2] = {make_float2(d.x, d.y), make_float2(d.z, d.w)};
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) h[k][s] = fma2(ex2_2(mul2(sum[k], A[k][s])), h[k][s], own[k][s]);
        }
    }
    float2 total[2] = {both(0.f), both(0.f)};   // steps so far

    for (int tile = 0; tile < tiles; ++tile) {
        if (tile + 1 < tiles) load(tile + 1);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();   // the tile has landed, and all warps are done with the one before
        const unsigned char* const raw = smem + (tile & 1) * S::kStage;
        const int first = t0 + tile * TT, count = min(TT, live - first);
#pragma unroll
        for (int i = 0; i < PIECES; i += 32) {
            const int piece = i + lane, r = piece / (WCH / V), c = warp * WCH + piece % (WCH / V) * V;
            if (piece < PIECES) {
                float uu[V], dd[V];
                const uint4* const at = reinterpret_cast<const uint4*>(raw + r * S::kRow + c * sizeof(E));
                unpack(at[0], uu, E{});
                unpack(at[TT * S::kRow / 16], dd, E{});
                const bool ok = r < count && c < w.count;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float v = dd[k] + bias[c + k];
                    dd[k] = ok ? p.softplus ? softplus(v) : v : 0.f;
                    uu[k] = ok ? dd[k] * uu[k] : 0.f;
                    dd[k] *= kLog2e;
                }
#pragma unroll
                for (int k = 0; k < V; k += 4) {
                    *reinterpret_cast<float4*>(steps + r * CH + c + k) = make_float4(dd[k], dd[k + 1], dd[k + 2], dd[k + 3]);
                    *reinterpret_cast<float4*>(xs + r * CH + c + k) = make_float4(uu[k], uu[k + 1], uu[k + 2], uu[k + 3]);
                }
            }
        }
        for (int i = threadIdx.x; i < (OUT ? 2 : 1) * TT * N / V; i += kThreads) {   // B, then C
            float v[V];
            unpack(reinterpret_cast<const uint4*>(raw + 3 * TT * S::kRow)[i], v, E{});
#pragma unroll
            for (int k = 0; k < V; k += 4)
                *reinterpret_cast<float4*>(Bf + i * V + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
        __syncthreads();
        for (int r = 0; r < count; r += 4) {
            float out[4];
#pragma unroll
            for (int q = 0; q < 4; ++q) {
                const float4 d = *reinterpret_cast<const float4*>(steps + (r + q) * CH + quad);
                const float4 x = *reinterpret_cast<const float4*>(xs + (r + q) * CH + quad);
                const float4 b = *reinterpret_cast<const float4*>(Bf + (r + q) * N + n4);
                const float2 dd[2] = {make_float2(d.x, d.y), make_float2(d.z, d.w)};
                const float2 xx[2] = {make_float2(x.x, x.y), make_float2(x.z, x.w)};
                const float2 bb[4] = {both(b.x), both(b.y), both(b.z), both(b.w)};
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int s = 0; s < 4; ++s) h[k][s] = fma2(ex2_2(mul2(dd[k], A[k][s])), h[k][s], mul2(xx[k], bb[s]));
                if constexpr (OUT) {
                    const float4 c = *reinterpret_cast<const float4*>(Cf + (r + q) * N + n4);
                    const float2 cc[4] = {both(c.x), both(c.y), both(c.z), both(c.w)};
                    float2 o[2];
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        o[k] = mul2(cc[0], h[k][0]);
#pragma unroll
                        for (int s = 1; s < 4; ++s) o[k] = fma2(cc[s], h[k][s], o[k]);
                    }
                    out[q] = quad_sum<L::kLanes>(o[0].x, o[0].y, o[1].x, o[1].y);
                } else {
                    total[0] = add2(total[0], dd[0]);
                    total[1] = add2(total[1], dd[1]);
                }
            }
            if constexpr (OUT) {
                __syncwarp();   // the outputs take their inputs' place
                if (quad_leader<L::kLanes>())
#pragma unroll
                    for (int q = 0; q < 4; ++q) xs[(r + q) * CH + quad + quad_channel<L::kLanes>()] = out[q];
            }
        }
        if constexpr (OUT) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PIECES; i += 32) {
                const int piece = i + lane, r = piece / (WCH / V), c = warp * WCH + piece % (WCH / V) * V;
                if (piece < PIECES && r < count && c < w.count) {
                    float uu[V], out[V];
                    const uint4* const at = reinterpret_cast<const uint4*>(raw + r * S::kRow + c * sizeof(E));
                    unpack(at[0], uu, E{});
#pragma unroll
                    for (int k = 0; k < V; ++k) out[k] = fmaf(skip[c + k], uu[k], xs[r * CH + c + k]);
                    if (gated) {
                        unpack(at[2 * TT * S::kRow / 16], uu, E{});
#pragma unroll
                        for (int k = 0; k < V; ++k) out[k] *= uu[k] * sigmoid(uu[k]);
                    }
                    store_vec<E>(y, static_cast<size_t>(first + r) * p.D + c, pack(out, E{}));
                }
            }
            __syncwarp();
        }
    }
    if constexpr (OUT) {
        if (w.segment == last && on && p.h_out) store_states(p.h_out + mat, N, h);
    } else if (on) {
        store_states(p.seg_state + w.segment * all + mat, N, h);
        if (n4 == 0)
            *reinterpret_cast<float4*>(p.seg_dt + (static_cast<size_t>(w.segment) * p.B + w.b) * p.D + w.first + quad) =
                make_float4(total[0].x, total[0].y, total[1].x, total[1].y);
    }
    cp_async_wait<0>();
}

// One token: a thread holds four states of one channel, so its N / 4 lanes sum y.
template <typename E, int N>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(const __grid_constant__ SsmParams p)
{
    constexpr int LANES = N / 4;
    const long long item = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const int c = static_cast<int>(item / LANES % p.D), n4 = static_cast<int>(item % LANES) * 4;
    const long long row = item / LANES / p.D;
    const bool on = row < p.B;
    const long long b = on ? row : 0;
    const int group = c / (p.D / p.G);
    const size_t mat = (static_cast<size_t>(b) * p.D + c) * N + n4;
    const float4 h = *reinterpret_cast<const float4*>(p.h_in + mat);
    const float4 A = __ldg(reinterpret_cast<const float4*>(p.A + static_cast<size_t>(c) * N + n4));
    const E* const Bt = static_cast<const E*>(p.Bt) + b * p.ld_bc + group * N + n4;
    const E* const Ct = static_cast<const E*>(p.Ct) + b * p.ld_bc + group * N + n4;
    const float u = to_f(static_cast<const E*>(p.u)[b * p.ld_u + c]);
    const float v = to_f(static_cast<const E*>(p.dt)[b * p.ld_dt + c]) + (p.dt_bias ? __ldg(p.dt_bias + c) : 0.f);
    const float s = p.softplus ? softplus(v) : v, x = s * u, d = s * kLog2e;
    float4 g;
    g.x = fmaf(ex2(d * A.x), h.x, x * to_f(Bt[0]));
    g.y = fmaf(ex2(d * A.y), h.y, x * to_f(Bt[1]));
    g.z = fmaf(ex2(d * A.z), h.z, x * to_f(Bt[2]));
    g.w = fmaf(ex2(d * A.w), h.w, x * to_f(Bt[3]));
    float o = fmaf(to_f(Ct[0]), g.x, to_f(Ct[1]) * g.y) + fmaf(to_f(Ct[2]), g.z, to_f(Ct[3]) * g.w);
#pragma unroll
    for (int k = LANES / 2; k > 0; k >>= 1) o += __shfl_xor_sync(0xffffffffu, o, k);
    if (!on) return;
    *reinterpret_cast<float4*>(p.h_out + mat) = g;
    if (n4 != 0) return;
    if (p.skip) o = fmaf(__ldg(p.skip + c), u, o);
    if (p.z) {
        const float z = to_f(static_cast<const E*>(p.z)[b * p.ld_z + c]);
        o *= z * sigmoid(z);
    }
    static_cast<E*>(p.y)[static_cast<size_t>(b) * p.D + c] = from_f<E>(o);
}

struct Plan {
    int segments, seg_len;
};

// Segments of whole tiles, where whole sequences would leave most of the SMs idle.
Plan plan_of(int B, int T, int D, int N, int G)
{
    const int ch = kWarps * 128 / (N / 4), dg = D / G;
    const long long ctas = static_cast<long long>(B) * G * ((dg + ch - 1) / ch);
    const int most = std::max(1, T / (4 * TT));
    const int segments = ctas >= 2 * kSms ? 1 : static_cast<int>(std::min<long long>(most, std::min<long long>(64, (4 * kSms + ctas - 1) / ctas)));
    if (segments <= 1) return {1, std::max(1, T)};
    const int tiles = (T + TT - 1) / TT, per = (tiles + segments - 1) / segments;
    return {(tiles + per - 1) / per, per * TT};
}

template <typename E, int N>
int forward(const SsmParams& p, cudaStream_t st)
{
    using S = Tile<E, N>;
    const int dg = p.D / p.G;
    const unsigned grid = static_cast<unsigned>(p.B) * p.G * ((dg + S::kCh - 1) / S::kCh);
    if (cudaFuncSetAttribute(ssm_kernel<E, N, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(ssm_kernel<E, N, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    if (p.segments > 1) {
        ssm_kernel<E, N, false><<<grid * (p.segments - 1), kThreads, S::kSmem, st>>>(p);
        const int rc = launched();
        if (rc != SRWM_OK) return rc;
    }
    ssm_kernel<E, N, true><<<grid * p.segments, kThreads, S::kSmem, st>>>(p);
    return launched();
}

template <typename E, int N>
int step(const SsmParams& p, cudaStream_t st)
{
    const long long items = static_cast<long long>(p.B) * p.D * (N / 4);
    ssm_step_kernel<E, N><<<static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
    return launched();
}

template <typename E>
int by_states(bool one, const SsmParams& p, cudaStream_t st)
{
    if (p.N == 16) return one ? step<E, 16>(p, st) : forward<E, 16>(p, st);
    if (p.N == 32) return one ? step<E, 32>(p, st) : forward<E, 32>(p, st);
    return one ? step<E, 64>(p, st) : forward<E, 64>(p, st);
}

int by_type(bool one, int dtype, const SsmParams& p, cudaStream_t st)
{
    if (dtype == SRWM_F32) return by_states<float>(one, p, st);
    if (dtype == SRWM_BF16) return by_states<__nv_bfloat16>(one, p, st);
    return by_states<__half>(one, p, st);
}

}  // namespace

size_t ssm_scratch(int B, int T, int D, int N, int G)
{
    const Plan plan = plan_of(B, T, D, N, G);
    return plan.segments > 1 ? round256(static_cast<size_t>(plan.segments) * B * D * (N + 1) * 4) : 256;
}

int ssm_launch(int dtype, SsmParams& p, void* workspace, cudaStream_t st)
{
    const Plan plan = plan_of(p.B, p.T, p.D, p.N, p.G);
    p.segments = plan.segments, p.seg_len = plan.seg_len;
    p.seg_state = static_cast<float*>(workspace);
    p.seg_dt = p.seg_state + static_cast<size_t>(plan.segments) * p.B * p.D * p.N;
    return by_type(false, dtype, p, st);
}

int ssm_step_launch(int dtype, const SsmParams& p, cudaStream_t st) { return by_type(true, dtype, p, st); }

}  // namespace srwm
