// srwm_ssm_bwd.cu -- gradients of the selective state space scan.
//
// With p_t = dy_t silu(z_t) (dy_t where there is no gate), a_t = exp(s_t A), x_t = s_t u_t and g_t = dL/dh_t:
//   g_t = C_t p_t + a_{t+1} g_{t+1}        (from dL/dh_final at the end)
//   q_t = a_t g_t h_{t-1},   e_t = sum_n g_t B_t
//   dC_t = sum_c p_t h_t,    dB_t = sum_c x_t g_t,    dA = sum q_t s_t
//   du_t = e_t s_t + skip p_t,   ds_t = sum_n q_t A + e_t u_t,   ddt_t = ds_t sigmoid(dt_t + dt_bias)
//   dz_t = dy_t (C_t . h_t + skip u_t) silu'(z_t),   dskip = sum p_t u_t,   ddt_bias = sum ddt_t
// A CTA (a range of channels, a sequence or a segment of it) runs its states forwards and leaves them at every
// tile's start in the workspace, then takes the tiles from the last to the first: forwards once more with the
// states before each token in shared memory, then backwards.  Nothing is divided by a decay, so strong decays lose
// nothing.  dB and dC leave as one partial per range of channels, the parameters' gradients as one per sequence
// (and segment); both are summed in a fixed order.
// Few streams: as in the forward pass, a first kernel runs every segment by itself, its states from zero and its
// gradient towards its start with nothing behind it; the second joins them.
#include <cuda_runtime.h>

#include <algorithm>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_ssm.cuh"
#include "srwm_sum.h"

namespace srwm {
namespace {

using namespace ssm;

constexpr int TT = 8;    // tokens of a tile
constexpr int kSms = 152;

enum Row { kU, kDt, kZ, kDy };

template <typename E, int N>
struct Tile {
    using L = Lay<N>;
    static constexpr int kCh = L::kCh;
    static constexpr int kRow = kCh * static_cast<int>(sizeof(E));
    static constexpr int kBc = N * static_cast<int>(sizeof(E));
    static constexpr int kStage = TT * (4 * kRow + 2 * kBc);          // u | dt | z | dy | B | C as they land
    static constexpr int kWide = TT * (5 * kCh + 2 * N) * 4;          // steps | inputs, e | p | sum q A | C . h | B | C
    static constexpr int kPart = kWarps * TT * 2 * N * 4;             // each warp's dB | dC
    static constexpr int kStates = TT * kThreads * 64;                // states before each token
    static constexpr int kFixed = 2 * kCh * 4;                        // dt_bias | skip
    static constexpr int kStages = sizeof(E) == 4 ? 1 : 2;
    static constexpr int kSmem = kStages * kStage + kWide + kPart + kStates + kFixed;
    static constexpr int kSmemLocal = 2 * kStage + TT * (3 * kCh + 2 * N) * 4 + kFixed;
};

// What both kernels have of their place and its rows.
template <typename E, int N>
struct Rows {
    Place w;
    int n, t0, t1, live, last;
    const E* row[4];
    long long ld[4];
    const E* bc[2];
    long long ld_bc;
    bool gated;

    __device__ __forceinline__ explicit Rows(const SsmParams& p) : w(place_of<Lay<N>::kCh>(p))
    {
        n = valid_tokens(p.lengths, w.b, p.T);
        t0 = w.segment * p.seg_len;
        t1 = min(p.T, t0 + p.seg_len);
        live = min(n, t1);
        last = n > 0 ? (n - 1) / p.seg_len : 0;
        const size_t tokens = static_cast<size_t>(w.b) * p.T;
        gated = p.z != nullptr;
        row[kU] = static_cast<const E*>(p.u) + tokens * p.ld_u + w.first;
        row[kDt] = static_cast<const E*>(p.dt) + tokens * p.ld_dt + w.first;
        row[kZ] = static_cast<const E*>(p.z) + (gated ? tokens * p.ld_z + w.first : 0);
        row[kDy] = static_cast<const E*>(p.dy) + tokens * p.D + w.first;
        ld[kU] = p.ld_u, ld[kDt] = p.ld_dt, ld[kZ] = p.ld_z, ld[kDy] = p.D;
        bc[0] = static_cast<const E*>(p.Bt) + tokens * p.ld_bc + w.group * N;
        bc[1] = static_cast<const E*>(p.Ct) + tokens * p.ld_bc + w.group * N;
        ld_bc = p.ld_bc;
    }

    // Tile `tile`'s rows to shared memory at `to`; WHOLE: all of them, else u, dt and B.  Zeros past the end.
    template <bool WHOLE>
    __device__ __forceinline__ void load(int tile, uint32_t to) const
    {
        using S = Tile<E, N>;
        using L = Lay<N>;
        constexpr int V = vec<E>, PIECES = TT * L::kWarpCh / V;
        const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, first = t0 + tile * TT;
#pragma unroll
        for (int k = 0; k < (WHOLE ? 4 : 2); ++k) {
            if (k == kZ && !gated) continue;
#pragma unroll
            for (int i = 0; i < PIECES; i += 32) {   // a warp's own channels
                const int piece = i + lane, r = piece / (L::kWarpCh / V), c = warp * L::kWarpCh + piece % (L::kWarpCh / V) * V;
                const bool ok = piece < PIECES && first + r < live && c < w.count;
                if (piece < PIECES)
                    cp_async16(to + k * TT * S::kRow + r * S::kRow + c * static_cast<int>(sizeof(E)),
                               row[k] + (ok ? static_cast<long long>(first + r) * ld[k] + c : 0), ok);
            }
        }
#pragma unroll
        for (int k = 0; k < (WHOLE ? 2 : 1); ++k)
            for (int i = threadIdx.x; i < TT * N / V; i += kThreads) {
                const int r = i / (N / V), c = i % (N / V) * V;
                const bool ok = first + r < live;
                cp_async16(to + 4 * TT * S::kRow + (k * TT + r) * S::kBc + c * static_cast<int>(sizeof(E)),
                           bc[k] + (ok ? static_cast<long long>(first + r) * ld_bc + c : 0), ok);
            }
    }
};

// A landed tile in fp32: steps (times log2 e) and inputs, and with WHOLE p; B, and with WHOLE C.
template <typename E, int N, bool WHOLE>
__device__ __forceinline__ void widen(const SsmParams& p, const Rows<E, N>& R, const unsigned char* raw, int count, const float* bias,
                                      float* steps, float* xs, float* ps, float* Bf)
{
    using S = Tile<E, N>;
    using L = Lay<N>;
    constexpr int V = vec<E>, PIECES = TT * L::kWarpCh / V, CH = S::kCh;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
#pragma unroll
    for (int i = 0; i < PIECES; i += 32) {
        const int piece = i + lane, r = piece / (L::kWarpCh / V), c = warp * L::kWarpCh + piece % (L::kWarpCh / V) * V;
        if (piece < PIECES) {
            float uu[V], dd[V];
            const uint4* const at = reinterpret_cast<const uint4*>(raw + r * S::kRow + c * sizeof(E));
            unpack(at[kU * TT * S::kRow / 16], uu, E{});
            unpack(at[kDt * TT * S::kRow / 16], dd, E{});
            const bool ok = r < count && c < R.w.count;
#pragma unroll
            for (int k = 0; k < V; ++k) {
                const float v = fmaf(dd[k], kLog2e, bias[c + k] * kLog2e);
                dd[k] = ok ? p.softplus ? softplus2(both(v)).x : v : 0.f;
                uu[k] = ok ? dd[k] * kLn2 * uu[k] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < V; k += 4) {
                *reinterpret_cast<float4*>(steps + r * CH + c + k) = make_float4(dd[k], dd[k + 1], dd[k + 2], dd[k + 3]);
                *reinterpret_cast<float4*>(xs + r * CH + c + k) = make_float4(uu[k], uu[k + 1], uu[k + 2], uu[k + 3]);
            }
            if constexpr (WHOLE) {
                unpack(at[kDy * TT * S::kRow / 16], uu, E{});
                if (R.gated) {
                    unpack(at[kZ * TT * S::kRow / 16], dd, E{});
#pragma unroll
                    for (int k = 0; k < V; ++k) uu[k] *= dd[k] * sigmoid(dd[k]);
                }
#pragma unroll
                for (int k = 0; k < V; k += 4)   // rows past the end came as zeros
                    *reinterpret_cast<float4*>(ps + r * CH + c + k) = make_float4(uu[k], uu[k + 1], uu[k + 2], uu[k + 3]);
            }
        }
    }
    for (int i = threadIdx.x; i < (WHOLE ? 2 : 1) * TT * N / V; i += kThreads) {
        float v[V];
        unpack(reinterpret_cast<const uint4*>(raw + 4 * TT * S::kRow)[i], v, E{});
#pragma unroll
        for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(Bf + i * V + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
    }
}

__device__ __forceinline__ void pairs(const float4& v, float2 (&r)[2]) { r[0] = make_float2(v.x, v.y), r[1] = make_float2(v.z, v.w); }
__device__ __forceinline__ void spread(const float4& v, float2 (&r)[4]) { r[0] = both(v.x), r[1] = both(v.y), r[2] = both(v.z), r[3] = both(v.w); }

// h = a h + x B
__device__ __forceinline__ void advance(const float2 (&dd)[2], const float2 (&xx)[2], const float2 (&bb)[4], const float2 (&A)[2][4], float2 (&h)[2][4])
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) h[k][s] = fma2(ex2_2(mul2(dd[k], A[k][s])), h[k][s], mul2(xx[k], bb[s]));
}

// Each segment by itself: its states' end from zero, the sum of its steps, and its gradient towards its start.
template <typename E, int N>
__global__ void __launch_bounds__(kThreads) ssm_local_kernel(const __grid_constant__ SsmParams p)
{
    using S = Tile<E, N>;
    using L = Lay<N>;
    constexpr int CH = S::kCh;
    extern __shared__ __align__(128) unsigned char smem[];
    float* const steps = reinterpret_cast<float*>(smem + 2 * S::kStage);
    float *const xs = steps + TT * CH, *const ps = xs + TT * CH, *const Bf = ps + TT * CH, *const Cf = Bf + TT * N;
    float* const bias = Cf + TT * N;
    const Rows<E, N> R(p);
    if (R.w.segment > R.last) return;
    for (int i = threadIdx.x; i < CH; i += kThreads) bias[i] = i < R.w.count && p.dt_bias ? p.dt_bias[R.w.first + i] : 0.f;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp * L::kWarpCh + lane / L::kLanes * 4, n4 = lane % L::kLanes * 4;
    const bool on = quad < R.w.count;
    const int tiles = R.live > R.t0 ? (R.live - R.t0 + TT - 1) / TT : 0;
    if (tiles > 0) R.template load<true>(0, smem_u32(smem));
    cp_async_commit();
    float2 A[2][4], h[2][4], g[2][4], far[2][4], total[2] = {both(0.f), both(0.f)};
    load_states(p.A + static_cast<size_t>(R.w.first + quad) * N + n4, N, on, A);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) h[k][s] = g[k][s] = both(0.f), far[k][s] = both(1.f);
    for (int tile = 0; tile < tiles; ++tile) {
        if (tile + 1 < tiles) R.template load<true>(tile + 1, smem_u32(smem) + ((tile + 1) & 1) * S::kStage);
        cp_async_commit();
        cp_async_wait<1>();
        __syncthreads();
        const int count = min(TT, R.live - R.t0 - tile * TT);
        widen<E, N, true>(p, R, smem + (tile & 1) * S::kStage, count, bias, steps, xs, ps, Bf);
        __syncthreads();
        for (int r = 0; r < count; ++r) {
            float2 dd[2], xx[2], pp[2], bb[4], cc[4];
            pairs(*reinterpret_cast<const float4*>(steps + r * CH + quad), dd);
            pairs(*reinterpret_cast<const float4*>(xs + r * CH + quad), xx);
            pairs(*reinterpret_cast<const float4*>(ps + r * CH + quad), pp);
            spread(*reinterpret_cast<const float4*>(Bf + r * N + n4), bb);
            spread(*reinterpret_cast<const float4*>(Cf + r * N + n4), cc);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                total[k] = add2(total[k], dd[k]);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float2 a = ex2_2(mul2(dd[k], A[k][s]));
                    h[k][s] = fma2(a, h[k][s], mul2(xx[k], bb[s]));
                    far[k][s] = mul2(far[k][s], a);
                    g[k][s] = fma2(far[k][s], mul2(cc[s], pp[k]), g[k][s]);
                }
            }
        }
    }
    cp_async_wait<0>();
    if (!on) return;
    const size_t at = (static_cast<size_t>(R.w.segment) * p.B + R.w.b) * p.D + R.w.first + quad;
    store_states(p.seg_state + at * N + n4, N, h);
    store_states(p.seg_grad + at * N + n4, N, g);
    if (n4 == 0) *reinterpret_cast<float4*>(p.seg_dt + at) = make_float4(total[0].x, total[0].y, total[1].x, total[1].y);
}

// dB and dC of one token: eight values of each lane, summed over the warp's channel quads.  Lane l ends with the
// 8 LANES / 32 values that start at result (l / LANES) * that, of [dB of the four states, dC of the four states].
template <int LANES>
__device__ __forceinline__ void quads_sum(float (&v)[8])
{
    int width = 8;
#pragma unroll
    for (int o = 16; o >= LANES; o >>= 1) {
        width >>= 1;
        const bool up = threadIdx.x & o;
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (i < width) {
                const float keep = up ? v[width + i] : v[i], give = up ? v[i] : v[width + i];
                v[i] = keep + __shfl_xor_sync(0xffffffffu, give, o);
            }
    }
}

template <typename E, int N>
__global__ void __launch_bounds__(kThreads) ssm_grad_kernel(const __grid_constant__ SsmParams p)
{
    using S = Tile<E, N>;
    using L = Lay<N>;
    constexpr int V = vec<E>, CH = S::kCh, WCH = L::kWarpCh, PIECES = TT * WCH / V;
    extern __shared__ __align__(128) unsigned char smem[];
    float4* const hs = reinterpret_cast<float4*>(smem) + threadIdx.x;   // [TT][4][threads]: this lane's states before each token
    unsigned char* const stages = smem + S::kStates;
    float* const steps = reinterpret_cast<float*>(stages + S::kStages * S::kStage);
    float *const xs = steps + TT * CH, *const ps = xs + TT * CH, *const qs = ps + TT * CH, *const ys = qs + TT * CH;
    float *const Bf = ys + TT * CH, *const Cf = Bf + TT * N;
    float* const part = Cf + TT * N;   // [warps][TT][2 N]
    float *const bias = part + kWarps * TT * 2 * N, *const skip = bias + CH;

    const Rows<E, N> R(p);
    const Place& w = R.w;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp * WCH + lane / L::kLanes * 4, n4 = lane % L::kLanes * 4;
    const bool on = quad < w.count;
    const size_t tokens = static_cast<size_t>(w.b) * p.T;
    E* const du = static_cast<E*>(p.du) + tokens * p.D + w.first;
    E* const ddt = static_cast<E*>(p.ddt) + tokens * p.D + w.first;
    E* const dz = static_cast<E*>(p.dz) + (R.gated ? tokens * p.ld_dz + w.first : 0);
    for (int i = threadIdx.x; i < (R.t1 - max(R.t0, R.live)) * (w.count / V); i += kThreads) {   // rows past the end
        const size_t t = max(R.t0, R.live) + i / (w.count / V);
        const int c = i % (w.count / V) * V;
        store_vec<E>(du, t * p.D + c, make_uint4(0, 0, 0, 0));
        store_vec<E>(ddt, t * p.D + c, make_uint4(0, 0, 0, 0));
        if (R.gated) store_vec<E>(dz, t * p.ld_dz + c, make_uint4(0, 0, 0, 0));
    }
    for (int i = threadIdx.x; i < CH; i += kThreads) {
        bias[i] = i < w.count && p.dt_bias ? p.dt_bias[w.first + i] : 0.f;
        skip[i] = i < w.count && p.skip ? p.skip[w.first + i] : 0.f;
    }
    const int tiles = R.live > R.t0 ? (R.live - R.t0 + TT - 1) / TT : 0;
    const uint32_t stage0 = smem_u32(stages);
    const size_t mat = (static_cast<size_t>(w.b) * p.D + w.first + quad) * N + n4, all = static_cast<size_t>(p.B) * p.D * N;
    float2 A[2][4], h[2][4], g[2][4], dA[2][4];
    load_states(p.A + static_cast<size_t>(w.first + quad) * N + n4, N, on, A);
    load_states(p.h_in + mat, N, on && p.h_in, h);
    load_states(p.dh_out + mat, N, on && p.dh_out, g);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) dA[k][s] = both(0.f);
    if (p.segments > 1 && w.segment <= R.last) {
        griddep_wait();
        auto join = [&](int j, const float* from, float2 (&v)[2][4]) {   // v = own + exp(A sum of steps) v
            float2 own[2][4], sum[2];
            load_states(from + j * all + mat, N, on, own);
            pairs(on ? *reinterpret_cast<const float4*>(p.seg_dt + (static_cast<size_t>(j) * p.B + w.b) * p.D + w.first + quad)
                     : make_float4(0.f, 0.f, 0.f, 0.f), sum);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) v[k][s] = fma2(ex2_2(mul2(sum[k], A[k][s])), v[k][s], own[k][s]);
        };
        for (int j = 0; j < w.segment; ++j) join(j, p.seg_state, h);
        for (int j = R.last; j > w.segment; --j) join(j, p.seg_grad, g);
    }
    // forwards: the states at every tile's start
    float* const check = p.check + (static_cast<size_t>(w.b) * ((p.T + TT - 1) / TT) + R.t0 / TT) * p.D * N +
                         static_cast<size_t>(w.first + quad) * N + n4;
    const size_t check_step = static_cast<size_t>(p.D) * N;
    for (int tile = 0; tile + 1 < tiles; ++tile) {
        __syncthreads();
        R.template load<false>(tile, stage0);
        cp_async_commit();
        cp_async_wait<0>();
        __syncthreads();
        widen<E, N, false>(p, R, stages, TT, bias, steps, xs, ps, Bf);
        __syncthreads();
        if (on) store_states(check + tile * check_step, N, h);
        for (int r = 0; r < TT; ++r) {
            float2 dd[2], xx[2], bb[4];
            pairs(*reinterpret_cast<const float4*>(steps + r * CH + quad), dd);
            pairs(*reinterpret_cast<const float4*>(xs + r * CH + quad), xx);
            spread(*reinterpret_cast<const float4*>(Bf + r * N + n4), bb);
            advance(dd, xx, bb, A, h);
        }
    }
    // backwards
    float dskip[V], dbias[V];
#pragma unroll
    for (int k = 0; k < V; ++k) dskip[k] = dbias[k] = 0.f;
    float* const bc_part = p.bc_part + ((static_cast<size_t>((w.first - w.group * (p.D / p.G)) / CH) * p.B * p.T + tokens) * p.G + w.group) * 2 * N;
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int count = min(TT, R.live - R.t0 - tile * TT);
        __syncthreads();
        R.template load<true>(tile, stage0);
        cp_async_commit();
        if (tile + 1 < tiles) load_states(check + tile * check_step, N, on, h);
        cp_async_wait<0>();
        __syncthreads();
        widen<E, N, true>(p, R, stages, count, bias, steps, xs, ps, Bf);
        __syncthreads();
        for (int r = 0; r < count; ++r) {
            float2 dd[2], xx[2], bb[4], cc[4];
            pairs(*reinterpret_cast<const float4*>(steps + r * CH + quad), dd);
            pairs(*reinterpret_cast<const float4*>(xs + r * CH + quad), xx);
            spread(*reinterpret_cast<const float4*>(Bf + r * N + n4), bb);
            spread(*reinterpret_cast<const float4*>(Cf + r * N + n4), cc);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; s += 2)
                    hs[(r * 4 + k * 2 + s / 2) * kThreads] = make_float4(h[k][s].x, h[k][s].y, h[k][s + 1].x, h[k][s + 1].y);
            advance(dd, xx, bb, A, h);
            if (R.gated) {
                float2 o[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    o[k] = mul2(cc[0], h[k][0]);
#pragma unroll
                    for (int s = 1; s < 4; ++s) o[k] = fma2(cc[s], h[k][s], o[k]);
                }
                const float v = quad_sum<L::kLanes>(o[0].x, o[0].y, o[1].x, o[1].y);
                if (quad_leader<L::kLanes>()) ys[r * CH + quad + quad_channel<L::kLanes>()] = v;
            }
        }
        for (int r = count - 1; r >= 0; --r) {
            float2 dd[2], xx[2], pp[2], bb[4], cc[4], e[2], qa[2];
            pairs(*reinterpret_cast<const float4*>(steps + r * CH + quad), dd);
            pairs(*reinterpret_cast<const float4*>(xs + r * CH + quad), xx);
            pairs(*reinterpret_cast<const float4*>(ps + r * CH + quad), pp);
            spread(*reinterpret_cast<const float4*>(Bf + r * N + n4), bb);
            spread(*reinterpret_cast<const float4*>(Cf + r * N + n4), cc);
            float2 before[2][4], db[4], dc[4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; s += 2) {
                    const float4 v = hs[(r * 4 + k * 2 + s / 2) * kThreads];
                    before[k][s] = make_float2(v.x, v.y), before[k][s + 1] = make_float2(v.z, v.w);
                }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    const float2 a = ex2_2(mul2(dd[k], A[k][s]));
                    const float2 here = fma2(cc[s], pp[k], g[k][s]);
                    g[k][s] = mul2(a, here);
                    const float2 q = mul2(g[k][s], before[k][s]);
                    dA[k][s] = fma2(q, dd[k], dA[k][s]);
                    qa[k] = s ? fma2(q, A[k][s], qa[k]) : mul2(q, A[k][s]);
                    e[k] = s ? fma2(here, bb[s], e[k]) : mul2(here, bb[s]);
                    db[s] = k ? fma2(here, xx[k], db[s]) : mul2(here, xx[k]);
                    dc[s] = k ? fma2(h[k][s], pp[k], dc[s]) : mul2(h[k][s], pp[k]);
                    h[k][s] = before[k][s];
                }
            float v[8];
#pragma unroll
            for (int s = 0; s < 4; ++s) v[s] = db[s].x + db[s].y, v[4 + s] = dc[s].x + dc[s].y;
            quads_sum<L::kLanes>(v);
            constexpr int WIDTH = L::kLanes / 4;   // values of a lane
            const int result = lane / L::kLanes * WIDTH;
#pragma unroll
            for (int i = 0; i < WIDTH; ++i) {
                const int j = result + i;   // of dB's four states, then dC's
                part[(warp * TT + r) * 2 * N + (j >= 4 ? N : 0) + n4 + j % 4] = v[i];
            }
            const float es = quad_sum<L::kLanes>(e[0].x, e[0].y, e[1].x, e[1].y);
            const float qq = quad_sum<L::kLanes>(qa[0].x, qa[0].y, qa[1].x, qa[1].y);
            __syncwarp();
            if (quad_leader<L::kLanes>()) {
                xs[r * CH + quad + quad_channel<L::kLanes>()] = es;
                qs[r * CH + quad + quad_channel<L::kLanes>()] = qq;
            }
        }
        __syncthreads();
        const int first = R.t0 + tile * TT;
        for (int i = threadIdx.x; i < count * 2 * N; i += kThreads) {
            const int r = i / (2 * N), j = i % (2 * N);
            float a = part[r * 2 * N + j];
#pragma unroll
            for (int k = 1; k < kWarps; ++k) a += part[(k * TT + r) * 2 * N + j];
            bc_part[static_cast<size_t>(first + r) * p.G * 2 * N + j] = a;
        }
#pragma unroll
        for (int i = 0; i < PIECES; i += 32) {
            const int piece = i + lane, r = piece / (WCH / V), c = warp * WCH + piece % (WCH / V) * V;
            if (piece < PIECES && r < count && c < w.count) {
                float uu[V], dd[V], out[V], sl[V];
                const uint4* const at = reinterpret_cast<const uint4*>(stages + r * S::kRow + c * sizeof(E));
                unpack(at[kU * TT * S::kRow / 16], uu, E{});
                unpack(at[kDt * TT * S::kRow / 16], dd, E{});
                const size_t t = first + r;
                const int at32 = r * CH + c;
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    const float pk = ps[at32 + k], es = xs[at32 + k];
                    out[k] = fmaf(es, steps[at32 + k] * kLn2, skip[c + k] * pk);
                    dskip[k] = fmaf(pk, uu[k], dskip[k]);
                    const float ds = fmaf(es, uu[k], qs[at32 + k]);
                    sl[k] = p.softplus ? ds * sigmoid(dd[k] + bias[c + k]) : ds;
                    dbias[k] += sl[k];
                }
                store_vec<E>(du, t * p.D + c, pack(out, E{}));
                store_vec<E>(ddt, t * p.D + c, pack(sl, E{}));
                if (R.gated) {
                    float zz[V];
                    unpack(at[kDy * TT * S::kRow / 16], dd, E{});
                    unpack(at[kZ * TT * S::kRow / 16], zz, E{});
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        const float s = sigmoid(zz[k]);
                        out[k] = dd[k] * fmaf(skip[c + k], uu[k], ys[at32 + k]) * s * fmaf(zz[k], 1.f - s, 1.f);
                    }
                    store_vec<E>(dz, t * p.ld_dz + c, pack(out, E{}));
                }
            }
        }
    }
    if (w.segment == 0 && on && p.dh_in) store_states(p.dh_in + mat, N, g);
    float* const params = p.part + (static_cast<size_t>(w.segment) * p.B + w.b) * p.D * (N + 2);
    if (on) {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < 4; ++s) dA[k][s] = mul2(dA[k][s], both(kLn2));
        store_states(params + static_cast<size_t>(w.first + quad) * N + n4, N, dA);
    }
    // a channel's sums over the rows that its lanes took
    constexpr int PER = WCH / V;   // lanes l, l + PER, ... have the same channels
#pragma unroll
    for (int k = 0; k < V; ++k) {
#pragma unroll
        for (int o = 16; o >= PER; o >>= 1) {
            dskip[k] += __shfl_xor_sync(0xffffffffu, dskip[k], o);
            dbias[k] += __shfl_xor_sync(0xffffffffu, dbias[k], o);
        }
    }
    if (lane < PER) {
        const int c = warp * WCH + lane * V;
        if (c < w.count)
#pragma unroll
            for (int k = 0; k < V; ++k) {
                params[static_cast<size_t>(p.D) * N + w.first + c + k] = dskip[k];
                params[static_cast<size_t>(p.D) * (N + 1) + w.first + c + k] = dbias[k];
            }
    }
}

// dB and dC: the partials' sums over the ranges of a group's channels; zeros past the end.
template <typename E>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const __grid_constant__ SsmParams p, int chan_tiles)
{
    griddep_wait();
    const int width = 2 * p.G * p.N;
    const long long rows = static_cast<long long>(p.B) * p.T, i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long token = i / (width / 4);
    if (token >= rows) return;
    const int j = static_cast<int>(i % (width / 4)) * 4, b = static_cast<int>(token / p.T), t = static_cast<int>(token % p.T);
    const int group = j / (2 * p.N), k = j % (2 * p.N);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < valid_tokens(p.lengths, b, p.T))
        for (int c = 0; c < chan_tiles; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(p.bc_part + (static_cast<size_t>(c) * rows + token) * width + j);
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
    E* const to = static_cast<E*>(k < p.N ? p.dB : p.dC) + token * p.ld_dbc + group * p.N + k % p.N;
    to[0] = from_f<E>(a.x), to[1] = from_f<E>(a.y), to[2] = from_f<E>(a.z), to[3] = from_f<E>(a.w);
}

struct Plan {
    int segments, seg_len, chan_tiles;
    long long ctas;   // of one segment
};

Plan plan_of(int B, int T, int D, int N, int G)
{
    const int ch = kWarps * 128 / (N / 4), dg = D / G;
    Plan plan{1, std::max(1, T), (dg + ch - 1) / ch, 0};
    plan.ctas = static_cast<long long>(B) * G * plan.chan_tiles;
    const int most = std::max(1, T / (8 * TT));
    const int segments = plan.ctas >= 2 * kSms ? 1 : static_cast<int>(std::min<long long>(most, std::min<long long>(64, (2 * kSms + plan.ctas - 1) / plan.ctas)));
    if (segments <= 1) return plan;
    const int tiles = (T + TT - 1) / TT, per = (tiles + segments - 1) / segments;
    plan.segments = (tiles + per - 1) / per;
    plan.seg_len = per * TT;
    return plan;
}

// The workspace's regions, in floats, and all of them in bytes.
struct Regions {
    size_t seg_state, seg_grad, seg_dt, check, bc_part, part, bytes;
};

Regions regions_of(const Plan& plan, int B, int T, int D, int N, int G)
{
    const size_t streams = static_cast<size_t>(B) * D;
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at += round256(floats * 4) / 4;
        return here;
    };
    Regions r{};
    const size_t seg = plan.segments > 1 ? plan.segments : 0;
    r.seg_state = take(seg * streams * N);
    r.seg_grad = take(seg * streams * N);
    r.seg_dt = take(seg * streams);
    r.check = take(static_cast<size_t>((T + TT - 1) / TT) * streams * N);
    r.bc_part = take(static_cast<size_t>(plan.chan_tiles) * B * T * G * 2 * N);
    r.part = take(static_cast<size_t>(plan.segments) * B * D * (N + 2));
    r.bytes = std::max<size_t>(256, at * 4);
    return r;
}

template <typename E, int N>
int backward(const SsmParams& p, const Plan& plan, cudaStream_t st)
{
    using S = Tile<E, N>;
    if (cudaFuncSetAttribute(ssm_grad_kernel<E, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmem) != cudaSuccess ||
        cudaFuncSetAttribute(ssm_local_kernel<E, N>, cudaFuncAttributeMaxDynamicSharedMemorySize, S::kSmemLocal) != cudaSuccess) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    const unsigned grid = static_cast<unsigned>(plan.ctas * plan.segments);
    int rc = SRWM_OK;
    if (plan.segments > 1) {
        ssm_local_kernel<E, N><<<grid, kThreads, S::kSmemLocal, st>>>(p);
        rc = launched();
        if (rc != SRWM_OK) return rc;
    }
    ssm_grad_kernel<E, N><<<grid, kThreads, S::kSmem, st>>>(p);
    rc = launched();
    if (rc != SRWM_OK) return rc;
    const long long quads = static_cast<long long>(p.B) * p.T * (2 * p.G * N / 4);
    if (quads > 0) rc = launch_behind(ssm_bc_kernel<E>, dim3(static_cast<unsigned>((quads + 255) / 256)), 256, 0, st, p, plan.chan_tiles);
    if (rc != SRWM_OK) return rc;
    const long long rows = static_cast<long long>(plan.segments) * p.B;
    return sum_launch({p.part, rows, {p.dA, p.dskip, p.ddt_bias}, {static_cast<long long>(p.D) * N, p.D, p.D}}, st);
}

template <typename E>
int by_states(const SsmParams& p, const Plan& plan, cudaStream_t st)
{
    return p.N == 16 ? backward<E, 16>(p, plan, st) : p.N == 32 ? backward<E, 32>(p, plan, st) : backward<E, 64>(p, plan, st);
}

}  // namespace

size_t ssm_backward_scratch(int B, int T, int D, int N, int G) { return regions_of(plan_of(B, T, D, N, G), B, T, D, N, G).bytes; }

int ssm_backward_launch(int dtype, SsmParams& p, void* workspace, cudaStream_t st)
{
    const Plan plan = plan_of(p.B, p.T, p.D, p.N, p.G);
    const Regions r = regions_of(plan, p.B, p.T, p.D, p.N, p.G);
    float* const base = static_cast<float*>(workspace);
    p.segments = plan.segments, p.seg_len = plan.seg_len;
    p.seg_state = base + r.seg_state, p.seg_grad = base + r.seg_grad, p.seg_dt = base + r.seg_dt;
    p.check = base + r.check, p.bc_part = base + r.bc_part, p.part = base + r.part;
    if (dtype == SRWM_F32) return by_states<float>(p, plan, st);
    if (dtype == SRWM_BF16) return by_states<__nv_bfloat16>(p, plan, st);
    return by_states<__half>(p, plan, st);
}

}  // namespace srwm
