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
// Few streams, or a last wave nearly empty: as in the forward pass, a first kernel runs every segment by itself, its
// states from zero and its gradient towards its start with nothing behind it; the second joins them.
//
// What bounds it: 17 fp32 operations and three exponentials for each token, channel and state (three forwards, two and a
// quarter forwards once more, the rest backwards), with issue around them and shared memory's rate near.  64 x 1024 tokens
// of 1024 channels of 16 states, gated, in bf16 take 1.22 ms: 948 MB of inputs and gradients and 0.7 GB of states and
// partial sums, written and read, the fp32 pipe at 48 %, shared memory at 64 %, 53 % of the issue slots, where a two-wide
// operation holds two.  States of every other token in shared memory, and 168
// registers, leave room for six CTAs of two warps on an SM (57 sequences: 1167 us; four with 250 registers: 1372).
#include <cuda_runtime.h>

#include <algorithm>
#include <type_traits>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_ssm.cuh"
#include "srwm_sum.h"

namespace srwm {
namespace {

using namespace ssm;

constexpr int TT = 8;           // tokens of a tile
constexpr int kBlock = 32;      // tiles after which the parameters' sums go out: short chains of additions
constexpr int kSms = 152;

enum Row { kU, kDt, kZ, kDy };

template <typename E, int N>
struct Tile {
    using L = Lay<N>;
    static constexpr int kCh = L::kCh;
    static constexpr int kPitch = kCh + 4;                            // floats of a token's channels: other banks than the next's
    static constexpr int kRow = kCh * static_cast<int>(sizeof(E));
    static constexpr int kBc = N * static_cast<int>(sizeof(E));
    static constexpr int kHalf = TT * (2 * kRow + kBc);               // u | dt | B as they land
    static constexpr int kStage = 2 * kHalf;                          // .. | z | dy | C
    static constexpr int kWide = TT * kPitch * 4;                     // a token's channels in fp32
    static constexpr int kWideBc = TT * 2 * N * 4;                    // B | C in fp32
    static constexpr int kStates = TT / 2 * kThreads * 64;            // states before every other token
    static constexpr int kSmem = kStates + 2 * kStage + 4 * kWide + kWideBc;
    static constexpr int kSmemLocal = 2 * kStage + 3 * kWide + kWideBc;
};

// What both kernels have of their place, its rows and the channels that a lane widens and stores.
template <typename E, int N>
struct Rows {
    static constexpr int V = vec<E>, WCH = Lay<N>::kWarpCh;
    static constexpr int PER = WCH / 4, PIECES = TT * PER;   // four channels a lane
    Place w;
    int n, t0, t1, live, last, mine, tiles;
    const E* row[4];
    long long ld[4];
    const E* bc[2];
    long long ld_bc;
    bool gated, softplus;
    float2 bias[2];   // in units of log 2

    __device__ __forceinline__ explicit Rows(const SsmParams& p) : w(place_of<Lay<N>::kCh>(p))
    {
        n = valid_tokens(p.lengths, w.b, p.T);
        t0 = w.segment * w.seg_len;
        t1 = min(p.T, t0 + w.seg_len);
        live = min(n, t1);
        last = n > 0 ? (n - 1) / w.seg_len : 0;
        tiles = live > t0 ? (live - t0 + TT - 1) / TT : 0;
        mine = (threadIdx.x >> 5) * WCH + (threadIdx.x & 31) % PER * 4;
        const size_t tokens = static_cast<size_t>(w.b) * p.T;
        gated = p.z != nullptr;
        softplus = p.softplus != 0;
        row[kU] = static_cast<const E*>(p.u) + tokens * p.ld_u + w.first;
        row[kDt] = static_cast<const E*>(p.dt) + tokens * p.ld_dt + w.first;
        row[kZ] = static_cast<const E*>(p.z) + (gated ? tokens * p.ld_z + w.first : 0);
        row[kDy] = static_cast<const E*>(p.dy) + tokens * p.D + w.first;
        ld[kU] = p.ld_u, ld[kDt] = p.ld_dt, ld[kZ] = p.ld_z, ld[kDy] = p.D;
        bc[0] = static_cast<const E*>(p.Bt) + tokens * p.ld_bc + w.group * N;
        bc[1] = static_cast<const E*>(p.Ct) + tokens * p.ld_bc + w.group * N;
        ld_bc = p.ld_bc;
#pragma unroll
        for (int k = 0; k < 2; ++k)
            bias[k] = mine < w.count && p.dt_bias ? mul2(*reinterpret_cast<const float2*>(p.dt_bias + w.first + mine + 2 * k), both(kLog2e)) : both(0.f);
    }

    // Where row kind k's tile, and B's or C's, begin within a stage.
    static __device__ __forceinline__ constexpr int row_at(int k) { return k / 2 * Tile<E, N>::kHalf + k % 2 * TT * Tile<E, N>::kRow; }
    static __device__ __forceinline__ constexpr int bc_at(int k) { return k * Tile<E, N>::kHalf + 2 * TT * Tile<E, N>::kRow; }

    // Tile `tile`'s rows to shared memory at `to`; WHOLE: all of them, else u, dt and B.  Zeros past the end and the channels.
    template <bool WHOLE>
    __device__ __forceinline__ void load(int tile, uint32_t to) const
    {
        using S = Tile<E, N>;
        const int lane = threadIdx.x & 31, first = t0 + tile * TT;
#pragma unroll
        for (int k = 0; k < (WHOLE ? 4 : 2); ++k) {
            if (k == kZ && !gated) continue;
#pragma unroll
            for (int i = 0; i < TT * WCH / V; i += 32) {   // a warp's own channels
                const int piece = i + lane, r = piece / (WCH / V), c = (threadIdx.x >> 5) * WCH + piece % (WCH / V) * V;
                const bool ok = piece < TT * WCH / V && first + r < live && c < w.count;
                if (piece < TT * WCH / V)
                    cp_async16(to + row_at(k) + r * S::kRow + c * static_cast<int>(sizeof(E)),
                               row[k] + (ok ? static_cast<long long>(first + r) * ld[k] + c : 0), ok);
            }
        }
#pragma unroll
        for (int k = 0; k < (WHOLE ? 2 : 1); ++k)
            for (int i = threadIdx.x; i < TT * N / V; i += kThreads) {
                const int r = i / (N / V), c = i % (N / V) * V;
                const bool ok = first + r < live;
                cp_async16(to + bc_at(k) + r * S::kBc + c * static_cast<int>(sizeof(E)),
                           bc[k] + (ok ? static_cast<long long>(first + r) * ld_bc + c : 0), ok);
            }
    }

    // Four values of row kind k, `at` the place within a row of the first kind.
    static __device__ __forceinline__ void get(const unsigned char* at, int k, float (&f)[4])
    {
        unpack_quad(*reinterpret_cast<const typename Quad<E>::type*>(at + row_at(k)), f, E{});
    }

    // A landed tile in fp32: steps (in units of log 2) and inputs (times 1 / log 2: B has the factor), and with WHOLE p; B
    // times log 2, and with WHOLE C.  Steps are 0 past the end.
    template <bool WHOLE>
    __device__ __forceinline__ void widen(int tile, const unsigned char* raw, float* steps, float* xs, float* ps, float* Bf) const
    {
        using S = Tile<E, N>;
        const int lane = threadIdx.x & 31, count = live - t0 - tile * TT;
#pragma unroll
        for (int i = 0; i < PIECES; i += 32) {
            const int piece = i + lane, r = piece / PER;
            if (piece < PIECES) {
                float uu[4], dd[4];
                const unsigned char* const at = raw + r * S::kRow + mine * static_cast<int>(sizeof(E));
                const int to = r * S::kPitch + mine;
                get(at, kU, uu);
                get(at, kDt, dd);
                float2 s0 = fma2(make_float2(dd[0], dd[1]), both(kLog2e), bias[0]);
                float2 s1 = fma2(make_float2(dd[2], dd[3]), both(kLog2e), bias[1]);
                if (softplus) s0 = softplus2(s0), s1 = softplus2(s1);
                if (r >= count) s0 = s1 = both(0.f);
                const float2 x0 = mul2(s0, make_float2(uu[0], uu[1])), x1 = mul2(s1, make_float2(uu[2], uu[3]));
                *reinterpret_cast<float4*>(steps + to) = make_float4(s0.x, s0.y, s1.x, s1.y);
                *reinterpret_cast<float4*>(xs + to) = make_float4(x0.x, x0.y, x1.x, x1.y);
                if constexpr (WHOLE) {   // rows past the end came as zeros
                    get(at, kDy, uu);
                    float2 p0 = make_float2(uu[0], uu[1]), p1 = make_float2(uu[2], uu[3]);
                    if (gated) {
                        get(at, kZ, dd);
                        p0 = mul2(silu(make_float2(dd[0], dd[1])), p0), p1 = mul2(silu(make_float2(dd[2], dd[3])), p1);
                    }
                    *reinterpret_cast<float4*>(ps + to) = make_float4(p0.x, p0.y, p1.x, p1.y);
                }
            }
        }
        for (int i = threadIdx.x; i < (WHOLE ? 2 : 1) * TT * N / V; i += kThreads) {
            float v[V];
            unpack(reinterpret_cast<const uint4*>(raw + bc_at(i >= TT * N / V))[i % (TT * N / V)], v, E{});
            if (i < TT * N / V)
#pragma unroll
                for (int k = 0; k < V; ++k) v[k] *= kLn2;
#pragma unroll
            for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(Bf + i * V + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
        }
    }
};

__device__ __forceinline__ void pairs(const float* from, float2 (&r)[2])
{
    const float4 v = *reinterpret_cast<const float4*>(from);
    r[0] = make_float2(v.x, v.y), r[1] = make_float2(v.z, v.w);
}
__device__ __forceinline__ void spread(const float* from, float2 (&r)[4])
{
    const float4 v = *reinterpret_cast<const float4*>(from);
    r[0] = both(v.x), r[1] = both(v.y), r[2] = both(v.z), r[3] = both(v.w);
}

// A token's decays, and h = a h + x B.
__device__ __forceinline__ void decays(const float2 (&dd)[2], const float2 (&A)[2][4], float2 (&a)[2][4])
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) a[k][s] = decay2(dd[k], A[k][s]);
}
__device__ __forceinline__ void advance(const float2 (&a)[2][4], const float2 (&xx)[2], const float2 (&bb)[4], const float2 (&from)[2][4], float2 (&h)[2][4])
{
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) h[k][s] = fma2(a[k][s], from[k][s], mul2(xx[k], bb[s]));
}

// Each segment by itself: its states' end from zero, the sum of its steps, and its gradient towards its start.
template <typename E, int N>
__global__ void __launch_bounds__(kThreads) ssm_local_kernel(const __grid_constant__ SsmParams p)
{
    using S = Tile<E, N>;
    using L = Lay<N>;
    extern __shared__ __align__(128) unsigned char smem[];
    float* const steps = reinterpret_cast<float*>(smem + 2 * S::kStage);
    float *const xs = steps + S::kWide / 4, *const ps = xs + S::kWide / 4, *const Bf = ps + S::kWide / 4, *const Cf = Bf + TT * N;
    const Rows<E, N> R(p);
    griddep_launch();   // the second kernel's CTAs find their places beside this one's
    if (R.w.segment > R.last) return;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int quad = warp * L::kWarpCh + lane / L::kLanes * 4, n4 = lane % L::kLanes * 4;
    const bool on = quad < R.w.count;
    if (R.tiles > 0) R.template load<true>(0, smem_u32(smem));
    cp_async_commit();
    float2 A[2][4], h[2][4], g[2][4], far[2][4], total[2] = {both(0.f), both(0.f)};
    load_states(p.A + static_cast<size_t>(R.w.first + quad) * N + n4, N, on, A);
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) h[k][s] = g[k][s] = both(0.f), far[k][s] = both(1.f);
    // where a decay can be above 1, far can be infinite, and a token without a gradient is to add nothing all the same
    // (14 x 1024 x 1024 channels bf16: 367 us either way, 375 with the question asked of every warp)
    bool grows = !R.softplus;
#pragma unroll
    for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int s = 0; s < 4; ++s) grows |= A[k][s].x > 0.f || A[k][s].y > 0.f;
    grows = __any_sync(0xffffffffu, grows);
    auto run = [&](auto careful) {   // a tile's tokens
#pragma unroll 2
        for (int r = 0; r < TT; ++r) {
            float2 dd[2], xx[2], pp[2], bb[4], cc[4], a[2][4];
            pairs(steps + r * S::kPitch + quad, dd);
            pairs(xs + r * S::kPitch + quad, xx);
            pairs(ps + r * S::kPitch + quad, pp);
            spread(Bf + r * N + n4, bb);
            spread(Cf + r * N + n4, cc);
            decays(dd, A, a);
            advance(a, xx, bb, h, h);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                total[k] = add2(total[k], dd[k]);
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    far[k][s] = mul2(far[k][s], a[k][s]);
                    const float2 c = mul2(cc[s], pp[k]);
                    if constexpr (decltype(careful)::value) {
                        if (c.x != 0.f) g[k][s].x = fmaf(far[k][s].x, c.x, g[k][s].x);
                        if (c.y != 0.f) g[k][s].y = fmaf(far[k][s].y, c.y, g[k][s].y);
                    } else {
                        g[k][s] = fma2(far[k][s], c, g[k][s]);
                    }
                }
            }
        }
    };
    for (int tile = 0; tile < R.tiles; ++tile) {
        cp_async_wait<0>();
        __syncthreads();   // the tile has landed, and all warps are done with the one before
        if (tile + 1 < R.tiles) R.template load<true>(tile + 1, smem_u32(smem) + ((tile + 1) & 1) * S::kStage);
        cp_async_commit();
        R.template widen<true>(tile, smem + (tile & 1) * S::kStage, steps, xs, ps, Bf);
        __syncthreads();
        if (grows)
            run(std::true_type{});
        else
            run(std::false_type{});
    }
    cp_async_wait<0>();
    if (!on) return;
    const size_t at = segment_at(p, R.w, R.w.segment) + quad;
    store_states(p.seg_state + at * N + n4, N, h);
    store_states(p.seg_grad + at * N + n4, N, g);
    if (n4 == 0) *reinterpret_cast<float4*>(p.seg_dt + at) = make_float4(total[0].x, total[0].y, total[1].x, total[1].y);
}

// Blocks of tiles of a whole sequence, and of a segment: each has a row of the parameters' partial sums.
struct Blocks {
    int whole, cut;
};

template <typename E, int N>
__global__ void __launch_bounds__(kThreads, sizeof(E) == 4 ? 4 : 6) ssm_grad_kernel(const __grid_constant__ SsmParams p, const Blocks count)
{
    using S = Tile<E, N>;
    using L = Lay<N>;
    constexpr int V = vec<E>, PER = Rows<E, N>::PER, PIECES = Rows<E, N>::PIECES, LANES = L::kLanes;
    extern __shared__ __align__(128) unsigned char smem[];
    // [TT / 2][4][threads]: this lane's states before every other token; then, in their place, two tokens' parts of dB and dC
    float4* const hs = reinterpret_cast<float4*>(smem) + threadIdx.x;
    unsigned char* const stages = smem + S::kStates;
    float* const steps = reinterpret_cast<float*>(stages + 2 * S::kStage);
    float *const xs = steps + S::kWide / 4, *const ps = xs + S::kWide / 4, *const ys = ps + S::kWide / 4;
    float *const Bf = ys + S::kWide / 4, *const Cf = Bf + TT * N;

    const Rows<E, N> R(p);
    const Place& w = R.w;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tiles = R.tiles, mine = R.mine;
    const int quad = warp * L::kWarpCh + lane / LANES * 4, n4 = lane % LANES * 4;
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
    float2 skip[2];
#pragma unroll
    for (int k = 0; k < 2; ++k)
        skip[k] = mine < w.count && p.skip ? *reinterpret_cast<const float2*>(p.skip + w.first + mine + 2 * k) : both(0.f);
    const uint32_t stage0 = smem_u32(stages);
    const size_t mat = (static_cast<size_t>(w.b) * p.D + w.first + quad) * N + n4;
    float2 A[2][4], h[2][4], g[2][4];
    load_states(p.A + static_cast<size_t>(w.first + quad) * N + n4, N, on, A);
    load_states(p.h_in + mat, N, on && p.h_in, h);
    load_states(p.dh_out + mat, N, on && p.dh_out, g);
    if (w.b >= p.whole && w.segment <= R.last) {
        griddep_wait();
        auto join = [&](int j, const float* from, float2 (&v)[2][4]) {   // v = own + exp(A sum of steps) v
            float2 own[2][4], sum[2];
            const size_t at = segment_at(p, w, j) + quad;
            load_states(from + at * N + n4, N, on, own);
            sum[0] = sum[1] = both(0.f);
            if (on) pairs(p.seg_dt + at, sum);
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) v[k][s] = past_segment(sum[k], A[k][s], v[k][s], own[k][s]);
        };
#pragma unroll 2
        for (int j = 0; j < w.segment; ++j) join(j, p.seg_state, h);
#pragma unroll 2
        for (int j = R.last; j > w.segment; --j) join(j, p.seg_grad, g);
    }
    // forwards: the states at every tile's start, and at the end
    float* const check = p.check + (static_cast<size_t>(w.b - p.base) * ((p.T + TT - 1) / TT) + R.t0 / TT) * p.D * N +
                         static_cast<size_t>(w.first + quad) * N + n4;
    const size_t check_step = static_cast<size_t>(p.D) * N;
#pragma unroll
    for (int tile = 0; tile < 3; ++tile) {   // four tiles of u, dt and B have room
        if (tile < tiles) R.template load<false>(tile, stage0 + tile * S::kHalf);
        cp_async_commit();
    }
    for (int tile = 0; tile < tiles; ++tile) {
        cp_async_wait<2>();
        __syncthreads();   // the tile has landed, and all warps are done with the one before
        if (tile + 3 < tiles) R.template load<false>(tile + 3, stage0 + ((tile + 3) & 3) * S::kHalf);
        cp_async_commit();
        R.template widen<false>(tile, stages + (tile & 3) * S::kHalf, steps, xs, ps, Bf);
        __syncthreads();
        if (on) store_states(check + tile * check_step, N, h);
#pragma unroll 2
        for (int r = 0; r < TT; ++r) {
            float2 dd[2], xx[2], bb[4], a[2][4];
            pairs(steps + r * S::kPitch + quad, dd);
            pairs(xs + r * S::kPitch + quad, xx);
            spread(Bf + r * N + n4, bb);
            decays(dd, A, a);
            advance(a, xx, bb, h, h);
        }
    }
    // backwards; h: the states after the tile
    __syncthreads();
    if (tiles > 0) R.template load<true>(tiles - 1, stage0 + ((tiles - 1) & 1) * S::kStage);
    cp_async_commit();
    const int blocks = w.b < p.whole ? count.whole : count.cut;
    float* const params = p.part + (w.b < p.whole ? static_cast<size_t>(w.b - p.base) * blocks : static_cast<size_t>(p.cut_row) +
                                    (static_cast<size_t>(w.segment) * (p.B - p.whole) + (w.b - p.whole)) * blocks) * p.D * (N + 2);
    const size_t param_step = static_cast<size_t>(p.D) * (N + 2);
    float2 dA[2][4], dskip[2], dbias[2];
    auto clear = [&]() {
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
            for (int s = 0; s < 4; ++s) dA[k][s] = both(0.f);
#pragma unroll
        for (int k = 0; k < 2; ++k) dskip[k] = dbias[k] = both(0.f);
    };
    auto flush = [&](int block) {   // a block's sums to its row of the partials
        float* const to = params + block * param_step;
        if (on) {
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) dA[k][s] = mul2(dA[k][s], both(kLn2));
            store_states(to + static_cast<size_t>(w.first + quad) * N + n4, N, dA);
        }
#pragma unroll
        for (int k = 0; k < 2; ++k) {   // lanes l, l + PER, ... have the same channels
#pragma unroll
            for (int o = 16; o >= PER; o >>= 1) {
                dskip[k].x += __shfl_xor_sync(0xffffffffu, dskip[k].x, o), dskip[k].y += __shfl_xor_sync(0xffffffffu, dskip[k].y, o);
                dbias[k].x += __shfl_xor_sync(0xffffffffu, dbias[k].x, o), dbias[k].y += __shfl_xor_sync(0xffffffffu, dbias[k].y, o);
            }
            if (lane < PER && mine < w.count) {
                *reinterpret_cast<float2*>(to + static_cast<size_t>(p.D) * N + w.first + mine + 2 * k) = dskip[k];
                *reinterpret_cast<float2*>(to + static_cast<size_t>(p.D) * (N + 1) + w.first + mine + 2 * k) = dbias[k];
            }
        }
        clear();
    };
    clear();
    for (int block = blocks - 1; block >= 0 && block * kBlock >= tiles; --block) flush(block);
    float* const bc_part = p.bc_part + ((static_cast<size_t>((w.first - w.group * (p.D / p.G)) / S::kCh) * p.span + (w.b - p.base)) * p.T * p.G + w.group) * 2 * N;
    float2 start[2][4];   // the states before the tile
    load_states(check + max(tiles - 1, 0) * check_step, N, on && tiles > 0, start);
    for (int tile = tiles - 1; tile >= 0; --tile) {
        const int first = R.t0 + tile * TT, rows = min(TT, R.live - first);
        const unsigned char* const raw = stages + (tile & 1) * S::kStage;
        cp_async_wait<0>();
        __syncthreads();
        if (tile > 0) R.template load<true>(tile - 1, stage0 + ((tile - 1) & 1) * S::kStage);
        cp_async_commit();
        R.template widen<true>(tile, raw, steps, xs, ps, Bf);
        __syncthreads();
#pragma unroll
        for (int j = 0; j < TT / 2; ++j) {   // forwards: the states before tokens 0, 2, ..
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; s += 2)
                    hs[(j * 4 + k * 2 + s / 2) * kThreads] = make_float4(start[k][s].x, start[k][s].y, start[k][s + 1].x, start[k][s + 1].y);
            if (j == TT / 2 - 1) break;
#pragma unroll
            for (int r = 2 * j; r < 2 * j + 2; ++r) {
                float2 dd[2], xx[2], bb[4], a[2][4];
                pairs(steps + r * S::kPitch + quad, dd);
                pairs(xs + r * S::kPitch + quad, xx);
                spread(Bf + r * N + n4, bb);
                decays(dd, A, a);
                advance(a, xx, bb, start, start);
            }
        }
#pragma unroll 2
        for (int j = TT / 2 - 1; j >= 0; --j) {   // backwards, two tokens at a time
            const int r = 2 * j;
            float2 before[2][4], between[2][4], a[2][4], dd[2], xx[2], bb[4];
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; s += 2) {
                    const float4 v = hs[(j * 4 + k * 2 + s / 2) * kThreads];
                    before[k][s] = make_float2(v.x, v.y), before[k][s + 1] = make_float2(v.z, v.w);
                }
            pairs(steps + r * S::kPitch + quad, dd);
            pairs(xs + r * S::kPitch + quad, xx);
            spread(Bf + r * N + n4, bb);
            decays(dd, A, a);
            advance(a, xx, bb, before, between);
            // one token backwards: `a` its decays, from and h the states before and after it
            auto back = [&](int t, const float2 (&da)[2][4], const float2 (&d)[2], const float2 (&x)[2], const float2 (&b)[4],
                            const float2 (&from)[2][4], const float2 (&after)[2][4], int slot) {
                float2 pp[2], cc[4], e[2], qa[2], o[2], db[4], dc[4];
                pairs(ps + t * S::kPitch + quad, pp);
                spread(Cf + t * N + n4, cc);
#pragma unroll
                for (int k = 0; k < 2; ++k)
#pragma unroll
                    for (int s = 0; s < 4; ++s) {
                        const float2 here = fma2(cc[s], pp[k], g[k][s]);
                        g[k][s] = mul2(da[k][s], here);
                        const float2 q = mul2(g[k][s], from[k][s]);
                        dA[k][s] = fma2(q, d[k], dA[k][s]);
                        qa[k] = s ? fma2(q, A[k][s], qa[k]) : mul2(q, A[k][s]);
                        e[k] = s ? fma2(here, b[s], e[k]) : mul2(here, b[s]);
                        o[k] = s ? fma2(after[k][s], cc[s], o[k]) : mul2(after[k][s], cc[s]);
                        db[s] = k ? fma2(here, x[k], db[s]) : mul2(here, x[k]);
                        dc[s] = k ? fma2(after[k][s], pp[k], dc[s]) : mul2(after[k][s], pp[k]);
                    }
                hs[(j * 4 + slot * 2) * kThreads] = make_float4(db[0].x + db[0].y, db[1].x + db[1].y, db[2].x + db[2].y, db[3].x + db[3].y);
                hs[(j * 4 + slot * 2 + 1) * kThreads] = make_float4(dc[0].x + dc[0].y, dc[1].x + dc[1].y, dc[2].x + dc[2].y, dc[3].x + dc[3].y);
                const float es = quad_sum<LANES>(e[0].x, e[0].y, e[1].x, e[1].y);
                const float qq = quad_sum<LANES>(qa[0].x, qa[0].y, qa[1].x, qa[1].y);
                const float oo = R.gated ? quad_sum<LANES>(o[0].x, o[0].y, o[1].x, o[1].y) : 0.f;
                __syncwarp();   // all lanes have read what these replace
                if (quad_leader<LANES>()) {
                    const int at = t * S::kPitch + quad + quad_channel<LANES>();
                    xs[at] = es;
                    ps[at] = qq;
                    ys[at] = oo;
                }
            };
            {
                float2 d1[2], x1[2], b1[4], a1[2][4];
                pairs(steps + (r + 1) * S::kPitch + quad, d1);
                pairs(xs + (r + 1) * S::kPitch + quad, x1);
                spread(Bf + (r + 1) * N + n4, b1);
                decays(d1, A, a1);
                back(r + 1, a1, d1, x1, b1, between, h, 1);
            }
            {   // the first token's operands once more: registers for them all along cost more (64 x 1024 x 1024 channels bf16: 2 to 5 %)
                float2 d0[2], x0[2], b0[4];
                pairs(steps + r * S::kPitch + quad, d0);
                pairs(xs + r * S::kPitch + quad, x0);
                spread(Bf + r * N + n4, b0);
                back(r, a, d0, x0, b0, before, between, 0);
            }
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
                for (int s = 0; s < 4; ++s) h[k][s] = before[k][s];
        }
        load_states(check + max(tile - 1, 0) * check_step, N, on && tile > 0, start);
        __syncthreads();
        // dB and dC of the tile: each of a token's 2 N sums runs over the CTA's channel quads
        for (int i = threadIdx.x; i < TT * 2 * LANES; i += kThreads) {
            const int lane4 = i % LANES, c = i / LANES % 2, r = i / (2 * LANES);   // four of B's states, then of C's
            const float4* const from = reinterpret_cast<const float4*>(smem) + (r / 2 * 4 + r % 2 * 2 + c) * kThreads + lane4;
            float2 lo = both(0.f), hi = both(0.f);
#pragma unroll
            for (int q = 0; q < kThreads / LANES; ++q) {
                const float4 v = from[(N == 16 ? q ^ c : q) * LANES];   // of 16 states: C's lanes one quad aside, in other banks
                lo = add2(lo, make_float2(v.x, v.y)), hi = add2(hi, make_float2(v.z, v.w));
            }
            if (c == 0) lo = mul2(lo, both(kLn2)), hi = mul2(hi, both(kLn2));
            if (r < rows)
                *reinterpret_cast<float4*>(bc_part + static_cast<size_t>(first + r) * p.G * 2 * N + c * N + lane4 * 4) = make_float4(lo.x, lo.y, hi.x, hi.y);
        }
#pragma unroll
        for (int i = 0; i < PIECES; i += 32) {
            const int piece = i + lane, r = piece / PER;
            if (piece < PIECES && r < rows && mine < w.count) {
                float uu[4], vv[4], yy[4], zz[4], o1[4], o2[4], o3[4];
                const unsigned char* const at = raw + r * S::kRow + mine * static_cast<int>(sizeof(E));
                R.get(at, kU, uu);
                R.get(at, kDt, vv);
                R.get(at, kDy, yy);
                if (R.gated) R.get(at, kZ, zz);
                const size_t t = first + r;
                const int here = r * S::kPitch + mine;
                float2 step[2], e[2], qa[2], o[2];   // e: times log 2, as B
                pairs(steps + here, step);
                pairs(xs + here, e);
                pairs(ps + here, qa);
                pairs(ys + here, o);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float2 u = make_float2(uu[2 * k], uu[2 * k + 1]), dy = make_float2(yy[2 * k], yy[2 * k + 1]);
                    float2 pk = dy;
                    if (R.gated) {
                        const float2 z = make_float2(zz[2 * k], zz[2 * k + 1]), f = add2(ex2_2(mul2(z, both(-kLog2e))), both(1.f));
                        const float2 sg = make_float2(rcp_approx(f.x), rcp_approx(f.y)), gate = mul2(z, sg);
                        pk = mul2(dy, gate);
                        // silu'(z) = sg + z sg (1 - sg)
                        const float2 slope = fma2(gate, fma2(sg, both(-1.f), both(1.f)), sg);
                        const float2 v = mul2(mul2(dy, fma2(skip[k], u, o[k])), slope);
                        o3[2 * k] = v.x, o3[2 * k + 1] = v.y;
                    }
                    dskip[k] = fma2(pk, u, dskip[k]);
                    const float2 v = fma2(e[k], step[k], mul2(skip[k], pk));
                    o1[2 * k] = v.x, o1[2 * k + 1] = v.y;
                    float2 ds = fma2(mul2(e[k], both(kLog2e)), u, qa[k]);
                    if (R.softplus) {   // sigmoid(dt + dt_bias)
                        const float2 a = fma2(make_float2(vv[2 * k], vv[2 * k + 1]), both(kLog2e), R.bias[k]);
                        const float2 f = add2(make_float2(ex2(-a.x), ex2(-a.y)), both(1.f));
                        ds = mul2(ds, make_float2(rcp_approx(f.x), rcp_approx(f.y)));
                    }
                    dbias[k] = add2(dbias[k], ds);
                    o2[2 * k] = ds.x, o2[2 * k + 1] = ds.y;
                }
                store_quad<E>(du, t * p.D + mine, pack_quad(o1, E{}));
                store_quad<E>(ddt, t * p.D + mine, pack_quad(o2, E{}));
                if (R.gated) store_quad<E>(dz, t * p.ld_dz + mine, pack_quad(o3, E{}));
            }
        }
        if (tile % kBlock == 0) flush(tile / kBlock);
    }
    cp_async_wait<0>();
    if (w.segment == 0 && on && p.dh_in) store_states(p.dh_in + mat, N, g);
    griddep_wait();   // no CTA of this kernel ends before the one in front of it has
}

// dB and dC: the partials' sums over the ranges of a group's channels; zeros past the end.
template <typename E>
__global__ void __launch_bounds__(256) ssm_bc_kernel(const __grid_constant__ SsmParams p, int chan_tiles)
{
    griddep_wait();
    const int width = 2 * p.G * p.N;
    const long long rows = static_cast<long long>(p.span) * p.T, i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
    const long long token = i / (width / 4);
    if (token >= rows) return;
    const int j = static_cast<int>(i % (width / 4)) * 4, b = p.base + static_cast<int>(token / p.T), t = static_cast<int>(token % p.T);
    const int group = j / (2 * p.N), k = j % (2 * p.N);
    float4 a = make_float4(0.f, 0.f, 0.f, 0.f);
    if (t < valid_tokens(p.lengths, b, p.T))
        for (int c = 0; c < chan_tiles; ++c) {
            const float4 v = *reinterpret_cast<const float4*>(p.bc_part + (static_cast<size_t>(c) * rows + token) * width + j);
            a.x += v.x, a.y += v.y, a.z += v.z, a.w += v.w;
        }
    E* const to = static_cast<E*>(k < p.N ? p.dB : p.dC) + (static_cast<long long>(b) * p.T + t) * p.ld_dbc + group * p.N + k % p.N;
    to[0] = from_f<E>(a.x), to[1] = from_f<E>(a.y), to[2] = from_f<E>(a.z), to[3] = from_f<E>(a.w);
}

struct Plan {
    Split split;
    Blocks blocks;
    int chan_tiles;
    int slice;              // whole sequences of one launch: the workspace holds the states and partials of these alone
    long long ctas;         // of a sequence (or of a segment)
    long long whole_rows, cut_rows;   // rows of the parameters' partial sums, of the whole sequences of a launch and of the others
};

constexpr double kSliceBytes = 2e9;   // of the workspace's arrays by sequence, or one wave's need where that is more

// Six CTAs on an SM, in fp32 four: with 255 registers no more fit, and with fewer (five, spilling none) 64 x 1024 x 1024
// channels take 1506 us instead of 1626, but 38 sequences, which fill a wave of four, 847 instead of 835 and 128 x 26 x 256
// 35.4 instead of 34.9.  Cut against whole, N x 1024 x 1024 channels bf16: 8 sequences (128
// CTAs) 229 and 599 us, 14 372 and 608, 20 714 and 816, 64 (of whose 1024 CTAs 112 are left over) 1222 and 1586.
Plan plan_of(size_t e, int B, int T, int D, int N, int G)
{
    const int ch = kWarps * 128 / (N / 4), dg = D / G;
    Plan plan{};
    plan.chan_tiles = (dg + ch - 1) / ch;
    plan.ctas = static_cast<long long>(G) * plan.chan_tiles;
    plan.split = split_of(B, plan.ctas, T, (e == 4 ? 4 : 6) * kSms, 6 * kSms, 0.5, TT, 4 * TT);
    auto blocks = [](int tokens) { return (std::max(1, tokens) + kBlock * TT - 1) / (kBlock * TT); };
    plan.blocks = {blocks(T), blocks(plan.split.seg_len)};
    // of one sequence: the states of every eighth token, dB's and dC's partials, the parameters'
    const double each = static_cast<double>((T + TT - 1) / TT) * D * N * 4 + static_cast<double>(T) * plan.chan_tiles * 8.0 * G * N +
                        static_cast<double>(plan.blocks.whole) * D * (N + 2) * 4;
    const long long wave = (6LL * kSms + plan.ctas - 1) / plan.ctas, room = static_cast<long long>(kSliceBytes / each);
    plan.slice = static_cast<int>(std::min<long long>(B, std::max(wave, room / wave * wave)));
    plan.whole_rows = static_cast<long long>(std::min(plan.slice, plan.split.whole)) * plan.blocks.whole;
    plan.cut_rows = static_cast<long long>(B - plan.split.whole) * plan.split.segments * plan.blocks.cut;
    return plan;
}

// The workspace's regions, in floats, and all of them in bytes.
struct Regions {
    size_t seg_state, seg_grad, seg_dt, check, bc_part, part, bytes;
};

Regions regions_of(const Plan& plan, int B, int T, int D, int N, int G)
{
    size_t at = 0;
    auto take = [&](size_t floats) {
        const size_t here = at;
        at += round256(floats * 4) / 4;
        return here;
    };
    Regions r{};
    const size_t cut = static_cast<size_t>(plan.split.segments) * (B - plan.split.whole) * D;
    r.seg_state = take(cut * N);
    r.seg_grad = take(cut * N);
    r.seg_dt = take(cut);
    const size_t held = std::max(plan.slice, B - plan.split.whole);   // sequences
    r.check = take(static_cast<size_t>((T + TT - 1) / TT) * held * D * N);
    r.bc_part = take(static_cast<size_t>(plan.chan_tiles) * held * T * G * 2 * N);
    const long long rows = plan.slice >= B ? plan.whole_rows + plan.cut_rows : std::max(plan.whole_rows, plan.cut_rows);
    r.part = take(static_cast<size_t>(rows) * D * (N + 2));
    r.bytes = std::max<size_t>(256, at * 4);
    return r;
}

template <typename E, int N>
int backward(const SsmParams& p, const Plan& plan, cudaStream_t st)
{
    using S = Tile<E, N>;
    static_assert(S::kSmem <= 48 * 1024 && S::kSmemLocal <= 48 * 1024, "more needs the kernels' attribute");
    const unsigned whole = static_cast<unsigned>(plan.ctas * p.whole), cut = static_cast<unsigned>(plan.ctas * (p.B - p.whole) * p.segments);
    int rc = SRWM_OK;
    if (cut > 0) {
        SsmParams q = p;
        q.first = static_cast<int>(whole);
        ssm_local_kernel<E, N><<<cut, kThreads, S::kSmemLocal, st>>>(q);
        rc = launched();
    }
    // one launch where the workspace holds all sequences; else a slice of whole ones at a time, and those that are cut; each
    // adds its parameters' sums to those before it
    const bool at_once = plan.slice >= p.B;
    for (int base = 0; base < p.B && rc == SRWM_OK;) {
        SsmParams q = p;
        const bool last = base >= p.whole;
        q.base = base, q.span = at_once ? p.B : last ? p.B - p.whole : std::min(plan.slice, p.whole - base);
        q.first = static_cast<int>(plan.ctas * base);
        q.cut_row = at_once ? plan.whole_rows : 0;
        const long long rows = at_once ? plan.whole_rows + plan.cut_rows : last ? plan.cut_rows : static_cast<long long>(q.span) * plan.blocks.whole;
        const unsigned grid = at_once ? whole + cut : last ? cut : static_cast<unsigned>(plan.ctas * q.span);
        if (cut > 0 && base == 0)
            rc = launch_behind(ssm_grad_kernel<E, N>, dim3(grid), kThreads, S::kSmem, st, q, plan.blocks);
        else {
            ssm_grad_kernel<E, N><<<grid, kThreads, S::kSmem, st>>>(q, plan.blocks);
            rc = launched();
        }
        const long long quads = static_cast<long long>(q.span) * p.T * (2 * p.G * N / 4);
        if (quads > 0 && rc == SRWM_OK)
            rc = launch_behind(ssm_bc_kernel<E>, dim3(static_cast<unsigned>((quads + 255) / 256)), 256, 0, st, q, plan.chan_tiles);
        if (rc == SRWM_OK)
            rc = sum_launch({p.part, rows, {p.dA, p.dskip, p.ddt_bias}, {static_cast<long long>(p.D) * N, p.D, p.D}, base > 0}, st);
        base += q.span;
    }
    return rc;
}

template <typename E>
int by_states(const SsmParams& p, const Plan& plan, cudaStream_t st)
{
    return p.N == 16 ? backward<E, 16>(p, plan, st) : p.N == 32 ? backward<E, 32>(p, plan, st) : backward<E, 64>(p, plan, st);
}

}  // namespace

size_t ssm_backward_scratch(int B, int T, int D, int N, int G)
{
    return std::max(regions_of(plan_of(4, B, T, D, N, G), B, T, D, N, G).bytes, regions_of(plan_of(2, B, T, D, N, G), B, T, D, N, G).bytes);
}

int ssm_backward_launch(int dtype, SsmParams& p, void* workspace, cudaStream_t st)
{
    const Plan plan = plan_of(dtype_bytes(dtype), p.B, p.T, p.D, p.N, p.G);
    const Regions r = regions_of(plan, p.B, p.T, p.D, p.N, p.G);
    float* const base = static_cast<float*>(workspace);
    p.whole = plan.split.whole, p.segments = plan.split.segments, p.seg_len = plan.split.seg_len;
    p.seg_state = base + r.seg_state, p.seg_grad = base + r.seg_grad, p.seg_dt = base + r.seg_dt;
    p.check = base + r.check, p.bc_part = base + r.bc_part, p.part = base + r.part;
    if (dtype == SRWM_F32) return by_states<float>(p, plan, st);
    if (dtype == SRWM_BF16) return by_states<__nv_bfloat16>(p, plan, st);
    return by_states<__half>(p, plan, st);
}

}  // namespace srwm
