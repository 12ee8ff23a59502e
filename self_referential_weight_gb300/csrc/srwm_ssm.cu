// srwm_ssm.cu -- the selective state space scan: prompts and single tokens.
//
//   s_t = softplus(dt_t + dt_bias),  h_t = exp(s_t A) h_{t-1} + s_t u_t B_t,
//   y_t = (C_t . h_t + skip u_t) silu(z_t)
// per channel, with N states each.  A CTA takes a range of channels of one
// sequence (or of a segment of it) in tiles of tokens: u, dt, z, B and C come
// by asynchronous copies a tile ahead; each warp forms its channels' steps and
// inputs in fp32, runs its states (in registers throughout) over the tile, and
// gates and stores the outputs.  Past a sequence's end a token's step is 0, which
// leaves the state as it is.
// Few streams, or a last wave nearly empty: the axis is cut into segments.  A first
// kernel runs every segment but the last from a zero state; the second starts each
// from the states before it, H = exp(A sum s) H + H', and writes y.
//
// What bounds it: four fp32 operations and one exponential for each token, channel
// and state, all in registers, and issue around them.  64 x 1024 tokens of 1024
// channels of 16 states, gated, in bf16 take 321 us: 545 MB at 1.7 TB/s, the fp32
// pipe at 48 % and 60 % of the issue slots, where a two-wide operation holds two.
// 2048 warps are 3.4 a scheduler, and those with four set the time.  Two warps a
// CTA against one or four: 343, 353 and 482 us; eight states of two channels a
// lane against four of four: 352 and 407.  A token in decoding is bound by
// memory: 512 x 1024 channels of 64 states in bf16 take 45 us, 6.0 TB/s.
#include <cuda_runtime.h>

#include <algorithm>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_ssm.cuh"

namespace srwm {
namespace {

using namespace ssm;

constexpr int kSms = 152;
constexpr int kWhole = 16;   // segments are multiples of this many tokens, whole tiles of either size
constexpr int kLaneCh = 2;   // as one float2 of their floats, and one shuffle between the two halves of a warp
constexpr int kPromptWarps = 2;
constexpr int kPromptThreads = 32 * kPromptWarps;

// A lane holds eight states of each of kLaneCh channels; the N / 8 lanes of these channels lie as far apart as the warp
// has such sets, so a load of states is the same address for neighbouring lanes.
template <typename E, int N>
struct Tile {
    static constexpr int TT = sizeof(E) == 4 ? 8 : 16;                        // tokens
    static constexpr int kLanes = N / 8, kSets = 32 / kLanes;
    static constexpr int kWarpCh = kLaneCh * kSets, kCh = kPromptWarps * kWarpCh;
    static constexpr int kRow = kCh * static_cast<int>(sizeof(E));            // bytes of a token's channels
    static constexpr int kBc = N * static_cast<int>(sizeof(E));               // and of its B (or C)
    static constexpr int kStage = TT * (3 * kRow + 2 * kBc);                  // u | dt | z | B | C as they land
    static constexpr int kPitch = kCh + 4;                                    // floats of a token's steps: other banks than the next's
    static constexpr int kWideBc = sizeof(E) == 4 ? 0 : TT * 2 * N * 4;
    static constexpr int kSmem = 2 * kStage + TT * 2 * kPitch * 4 + kWideBc;  // steps | inputs (then outputs) | B | C in fp32
};

// The eight states of a channel from `from` on, as pairs.
__device__ __forceinline__ void load8(const float* from, bool on, float2 (&h)[4])
{
    const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
    const float4 a = on ? *reinterpret_cast<const float4*>(from) : zero, b = on ? *reinterpret_cast<const float4*>(from + 4) : zero;
    h[0] = make_float2(a.x, a.y), h[1] = make_float2(a.z, a.w), h[2] = make_float2(b.x, b.y), h[3] = make_float2(b.z, b.w);
}
__device__ __forceinline__ void store8(float* to, const float2 (&h)[4])
{
    *reinterpret_cast<float4*>(to) = make_float4(h[0].x, h[0].y, h[1].x, h[1].y);
    *reinterpret_cast<float4*>(to + 4) = make_float4(h[2].x, h[2].y, h[3].x, h[3].y);
}

// A lane's neighbouring channels.
__device__ __forceinline__ void load_ch(const float* from, float (&v)[kLaneCh])
{
    const float2 q = *reinterpret_cast<const float2*>(from);
    v[0] = q.x, v[1] = q.y;
}

// What one token takes from shared memory.
template <bool OUT>
struct Token {
    float d[kLaneCh], x[kLaneCh];
    float2 b[4], c[4];

    __device__ __forceinline__ void load(const float* step, const float* input, const float* B, const float* C)
    {
        load_ch(step, d);
        load_ch(input, x);
        load8(B, true, b);
        if (OUT) load8(C, true, c);
    }
};

template <typename E, int N, bool OUT>
__global__ void __launch_bounds__(kPromptThreads, 7) ssm_kernel(const __grid_constant__ SsmParams p)
{
    using S = Tile<E, N>;
    constexpr int V = vec<E>, TT = S::TT, WCH = S::kWarpCh;
    constexpr int PIECES = TT * WCH / V;   // of a warp's tile
    extern __shared__ __align__(128) unsigned char smem[];
    float* const steps = reinterpret_cast<float*>(smem + 2 * S::kStage);
    float* const xs = steps + TT * S::kPitch;
    float* const bcs = xs + TT * S::kPitch;   // B and C in fp32 (of 16 bits)

    const Place w = place_of<S::kCh>(p);
    const int n = valid_tokens(p.lengths, w.b, p.T);
    const int t0 = w.segment * w.seg_len, t1 = min(p.T, t0 + w.seg_len), live = min(n, t1);
    const int last = n > 0 ? (n - 1) / w.seg_len : 0;   // the segment at whose end the sequence ends
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int own = warp * WCH + lane % S::kSets * kLaneCh, n8 = lane / S::kSets * 8;   // this lane's channels and states
    const bool on = own < w.count;
    if (!OUT) {
        griddep_launch();   // the second kernel's CTAs find their places beside this one's
        if (w.segment >= last) return;   // nothing comes after it
    }

    E* const y = static_cast<E*>(p.y) + static_cast<size_t>(w.b) * p.T * p.D + w.first;
    if constexpr (OUT)   // rows past the end
        for (int i = threadIdx.x; i < (t1 - max(t0, live)) * (w.count / V); i += kPromptThreads)
            store_vec<E>(y, static_cast<size_t>(max(t0, live) + i / (w.count / V)) * p.D + i % (w.count / V) * V, make_uint4(0, 0, 0, 0));
    if (w.segment > last) {
        griddep_wait();
        return;
    }

    // the channels that this lane widens and stores, in every tile
    const int mine = warp * WCH + lane % (WCH / V) * V;
    float bias[V], skip[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        bias[k] = mine < w.count && p.dt_bias ? p.dt_bias[w.first + mine + k] * kLog2e : 0.f;
        skip[k] = mine < w.count && p.skip ? p.skip[w.first + mine + k] : 0.f;
    }
    const size_t tokens = static_cast<size_t>(w.b) * p.T;
    const E* const rows[3] = {static_cast<const E*>(p.u) + tokens * p.ld_u + w.first,
                              static_cast<const E*>(p.dt) + tokens * p.ld_dt + w.first,
                              static_cast<const E*>(p.z) + (p.z ? tokens * p.ld_z + w.first : 0)};
    const long long lds[3] = {p.ld_u, p.ld_dt, p.ld_z};
    const E* const bc[2] = {static_cast<const E*>(p.Bt) + tokens * p.ld_bc + w.group * N,
                            static_cast<const E*>(p.Ct) + tokens * p.ld_bc + w.group * N};
    const bool gated = OUT && p.z;
    auto load = [&](int tile) {   // zeros past the end and past the channels
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
            for (int i = threadIdx.x; i < TT * N / V; i += kPromptThreads) {
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

    const size_t mat = (static_cast<size_t>(w.b) * p.D + w.first + own) * N + n8;
    float2 A[kLaneCh][4], h[kLaneCh][4];
#pragma unroll
    for (int c = 0; c < kLaneCh; ++c) {
        load8(p.A + static_cast<size_t>(w.first + own + c) * N + n8, on, A[c]);
        load8(p.h_in + mat + c * N, OUT && on && p.h_in, h[c]);
    }
    if (OUT && w.segment > 0) {
        griddep_wait();
        for (int j = 0; j < w.segment; ++j) {
            float sum[kLaneCh] = {};
            const size_t at = segment_at(p, w, j) + own;
            if (on) load_ch(p.seg_dt + at, sum);
#pragma unroll
            for (int c = 0; c < kLaneCh; ++c) {
                float2 part[4];
                load8(p.seg_state + (at + c) * N + n8, on, part);
#pragma unroll
                for (int s = 0; s < 4; ++s) h[c][s] = past_segment(both(sum[c]), A[c][s], h[c][s], part[s]);
            }
        }
    }
    float total[kLaneCh] = {};   // steps so far

    for (int tile = 0; tile < tiles; ++tile) {
        cp_async_wait<0>();
        __syncthreads();   // the tile has landed, and all warps are done with the one before
        if (tile + 1 < tiles) load(tile + 1);
        cp_async_commit();
        const unsigned char* const raw = smem + (tile & 1) * S::kStage;
        const int first = t0 + tile * TT, count = min(TT, live - first);
#pragma unroll
        for (int i = 0; i < PIECES; i += 32) {
            const int piece = i + lane, r = piece / (WCH / V);
            if (piece < PIECES) {
                float uu[V], dd[V];
                const uint4* const at = reinterpret_cast<const uint4*>(raw + r * S::kRow + mine * sizeof(E));
                unpack(at[0], uu, E{});
                unpack(at[TT * S::kRow / 16], dd, E{});
#pragma unroll
                for (int k = 0; k < V; k += 4) {
                    float2 s0 = fma2(make_float2(dd[k], dd[k + 1]), both(kLog2e), make_float2(bias[k], bias[k + 1]));
                    float2 s1 = fma2(make_float2(dd[k + 2], dd[k + 3]), both(kLog2e), make_float2(bias[k + 2], bias[k + 3]));
                    if (p.softplus) s0 = softplus2(s0), s1 = softplus2(s1);
                    if (r >= count) s0 = s1 = both(0.f);
                    float2 x0 = mul2(s0, make_float2(uu[k], uu[k + 1])), x1 = mul2(s1, make_float2(uu[k + 2], uu[k + 3]));
                    if (sizeof(E) == 4) x0 = mul2(x0, both(kLn2)), x1 = mul2(x1, both(kLn2));   // else B has the factor
                    *reinterpret_cast<float4*>(steps + r * S::kPitch + mine + k) = make_float4(s0.x, s0.y, s1.x, s1.y);
                    *reinterpret_cast<float4*>(xs + r * S::kPitch + mine + k) = make_float4(x0.x, x0.y, x1.x, x1.y);
                }
            }
        }
        if constexpr (sizeof(E) == 2) {
            for (int i = threadIdx.x; i < (OUT ? 2 : 1) * TT * N / V; i += kPromptThreads) {
                float v[V];
                unpack(reinterpret_cast<const uint4*>(raw + 3 * TT * S::kRow)[i], v, E{});
                if (i < TT * N / V)
#pragma unroll
                    for (int k = 0; k < V; ++k) v[k] *= kLn2;
#pragma unroll
                for (int k = 0; k < V; k += 4) *reinterpret_cast<float4*>(bcs + i * V + k) = make_float4(v[k], v[k + 1], v[k + 2], v[k + 3]);
            }
            __syncthreads();
        } else {
            __syncwarp();
        }
        const float* const B8 = (sizeof(E) == 4 ? reinterpret_cast<const float*>(raw + 3 * TT * S::kRow) : bcs) + n8;
        const float* const C8 = B8 + TT * N;
        Token<OUT> now, next;
        now.load(steps + own, xs + own, B8, C8);
        auto token = [&](int r, int ahead) {
            next.load(steps + ahead * S::kPitch + own, xs + ahead * S::kPitch + own, B8 + ahead * N, C8 + ahead * N);
            float o[kLaneCh];
#pragma unroll
            for (int c = 0; c < kLaneCh; ++c) {
                const float2 d = both(now.d[c]), x = both(now.x[c]);
                float2 sum;
#pragma unroll
                for (int s = 0; s < 4; ++s) {
                    h[c][s] = fma2(decay2(d, A[c][s]), h[c][s], mul2(x, now.b[s]));
                    if (OUT) sum = s ? fma2(now.c[s], h[c][s], sum) : mul2(now.c[s], h[c][s]);
                }
                if (OUT) o[c] = sum.x + sum.y;
                if (!OUT) total[c] += now.d[c];
            }
            if constexpr (OUT) {   // the channels' sums over their lanes: each half of these takes one of the two
                const bool up = lane & 16;
                float v = (up ? o[1] : o[0]) + __shfl_xor_sync(0xffffffffu, up ? o[0] : o[1], 16);
#pragma unroll
                for (int k = 8; k >= S::kSets; k >>= 1) v += __shfl_xor_sync(0xffffffffu, v, k);
                // in their inputs' place, which all lanes have read
                if (S::kSets == 16 || (lane & 15) < S::kSets) xs[r * S::kPitch + own + up] = v;
            }
            now = next;
        };
        if (count == TT) {
#pragma unroll
            for (int r = 0; r < TT; ++r) token(r, r + 1 < TT ? r + 1 : r);
        } else {
#pragma unroll 1
            for (int r = 0; r < count; ++r) token(r, min(r + 1, TT - 1));
        }
        if constexpr (OUT) {
            __syncwarp();
#pragma unroll
            for (int i = 0; i < PIECES; i += 32) {
                const int piece = i + lane, r = piece / (WCH / V);
                if (piece < PIECES && r < count && mine < w.count) {
                    float uu[V], out[V];
                    const uint4* const at = reinterpret_cast<const uint4*>(raw + r * S::kRow + mine * sizeof(E));
                    unpack(at[0], uu, E{});
#pragma unroll
                    for (int k = 0; k < V; k += 4) {
                        const float4 o = *reinterpret_cast<const float4*>(xs + r * S::kPitch + mine + k);
                        const float2 v0 = fma2(make_float2(skip[k], skip[k + 1]), make_float2(uu[k], uu[k + 1]), make_float2(o.x, o.y));
                        const float2 v1 = fma2(make_float2(skip[k + 2], skip[k + 3]), make_float2(uu[k + 2], uu[k + 3]), make_float2(o.z, o.w));
                        out[k] = v0.x, out[k + 1] = v0.y, out[k + 2] = v1.x, out[k + 3] = v1.y;
                    }
                    if (gated) {
                        unpack(at[2 * TT * S::kRow / 16], uu, E{});
#pragma unroll
                        for (int k = 0; k < V; k += 2) {
                            const float2 v = mul2(silu(make_float2(uu[k], uu[k + 1])), make_float2(out[k], out[k + 1]));
                            out[k] = v.x, out[k + 1] = v.y;
                        }
                    }
                    store_vec<E>(y, static_cast<size_t>(first + r) * p.D + mine, pack(out, E{}));
                }
            }
            __syncwarp();
        }
    }
    if constexpr (OUT) {
        if (w.segment == last && on && p.h_out)
#pragma unroll
            for (int c = 0; c < kLaneCh; ++c) store8(p.h_out + mat + c * N, h[c]);
    } else if (on) {
#pragma unroll
        for (int c = 0; c < kLaneCh; ++c) store8(p.seg_state + (segment_at(p, w, w.segment) + own + c) * N + n8, h[c]);
        if (n8 == 0)
#pragma unroll
            for (int c = 0; c < kLaneCh; ++c) p.seg_dt[segment_at(p, w, w.segment) + own + c] = total[c];
    }
    cp_async_wait<0>();
    if (OUT) griddep_wait();   // no CTA of the second kernel ends before the first kernel has
}

// One token: a lane holds four states of each of four channels (as srwm_ssm.cuh) for ROWS sequences, all of whose loads are
// on their way at once.  Each lane forms one channel's step and input, which the others get by shuffles.
template <typename E, int N, int ROWS>
__global__ void __launch_bounds__(kThreads) ssm_step_kernel(const __grid_constant__ SsmParams p)
{
    constexpr int LANES = N / 4;
    const int items = p.D / 4 * LANES, sets = (p.B + ROWS - 1) / ROWS;
    const long long item = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const long long set = item / items;
    if (__all_sync(0xffffffffu, set >= sets)) return;
    const int at = static_cast<int>(item % items), quad = at / LANES * 4, n4 = at % LANES * 4, own = quad + quad_channel<LANES>();
    const int group = quad / (p.D / p.G);
    const bool live = set < sets;
    const size_t first = live ? set : 0;
    const E* const u0 = static_cast<const E*>(p.u) + first * p.ld_u + own;
    const E* const d0 = static_cast<const E*>(p.dt) + first * p.ld_dt + own;
    const E* const z0 = static_cast<const E*>(p.z) + (p.z ? first * p.ld_z + own : 0);
    const size_t bc = first * p.ld_bc + group * N + n4, mat = (first * p.D + quad) * N + n4;
    float2 A[2][4], h[ROWS][2][4];
    typename Quad<E>::type B[ROWS], C[ROWS];
    float u[ROWS], v[ROWS], z[ROWS];
    bool on[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        on[i] = live && set + i * sets < p.B;
        const size_t skip = on[i] ? static_cast<size_t>(i) * sets : 0;   // sequences between this and the thread's first
        load_states(p.h_in + mat + skip * p.D * N, N, true, h[i]);
        B[i] = load_quad<E>(p.Bt, bc + skip * p.ld_bc);
        C[i] = load_quad<E>(p.Ct, bc + skip * p.ld_bc);
        u[i] = to_f(u0[skip * p.ld_u]);
        v[i] = to_f(d0[skip * p.ld_dt]);
        z[i] = p.z ? to_f(z0[skip * p.ld_z]) : 0.f;
    }
    load_states(p.A + static_cast<size_t>(quad) * N + n4, N, true, A);
    const float bias = p.dt_bias ? __ldg(p.dt_bias + own) * kLog2e : 0.f, skip = p.skip ? __ldg(p.skip + own) : 0.f;
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
        const float a = fmaf(v[i], kLog2e, bias);
        const float d = p.softplus ? softplus2(both(a)).x : a, x = d * kLn2 * u[i];
        float dk[4], xk[4], bk[4], ck[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            dk[k] = __shfl_sync(0xffffffffu, d, k * (LANES / 4), LANES);
            xk[k] = __shfl_sync(0xffffffffu, x, k * (LANES / 4), LANES);
        }
        unpack_quad(B[i], bk, E{});
        unpack_quad(C[i], ck, E{});
        float2 o[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const float2 dd = make_float2(dk[2 * k], dk[2 * k + 1]), xx = make_float2(xk[2 * k], xk[2 * k + 1]);
#pragma unroll
            for (int s = 0; s < 4; ++s) {
                h[i][k][s] = fma2(decay2(dd, A[k][s]), h[i][k][s], mul2(xx, both(bk[s])));
                o[k] = s ? fma2(both(ck[s]), h[i][k][s], o[k]) : mul2(both(ck[s]), h[i][k][s]);
            }
        }
        float y = quad_sum<LANES>(o[0].x, o[0].y, o[1].x, o[1].y);
        if (!on[i]) continue;
        const size_t b = first + static_cast<size_t>(i) * sets;
        store_states(p.h_out + mat + static_cast<size_t>(i) * sets * p.D * N, N, h[i]);
        if (!quad_leader<LANES>()) continue;
        y = fmaf(skip, u[i], y);
        if (p.z) y *= z[i] * sigmoid(z[i]);
        static_cast<E*>(p.y)[b * p.D + own] = from_f<E>(y);
    }
}

// Eight CTAs on an SM, of which segments fill half (2 x 8192 x 1024 channels fp32: 148 us with 19 segments, 152 with 27, 154
// with 37: each starts from those before it).  Cut against whole: 8 x 1024 x 1024 channels bf16 (128 CTAs) 88 and 124 us, 14
// sequences (224) 144 and 130.
Split plan_of(int B, int T, int D, int N, int G)
{
    const int ch = kPromptWarps * kLaneCh * 256 / N, dg = D / G;
    return split_of(B, static_cast<long long>(G) * ((dg + ch - 1) / ch), T, 8 * kSms, 4 * kSms, 0.14, kWhole, 2 * kWhole);
}

template <typename E, int N>
int forward(const SsmParams& p, cudaStream_t st)
{
    using S = Tile<E, N>;
    const int dg = p.D / p.G;
    const unsigned ctas = static_cast<unsigned>(p.G) * ((dg + S::kCh - 1) / S::kCh), split = ctas * (p.B - p.whole);
    static_assert(S::kSmem <= 48 * 1024, "more needs the kernels' attribute");
    if (split > 0) {
        SsmParams q = p;
        q.first = static_cast<int>(ctas * p.whole);
        ssm_kernel<E, N, false><<<split * (p.segments - 1), kPromptThreads, S::kSmem, st>>>(q);
        const int rc = launched();
        if (rc != SRWM_OK) return rc;
    }
    const unsigned grid = ctas * p.whole + split * p.segments;
    if (split > 0) return launch_behind(ssm_kernel<E, N, true>, dim3(grid), kPromptThreads, S::kSmem, st, p);
    ssm_kernel<E, N, true><<<grid, kPromptThreads, S::kSmem, st>>>(p);
    return launched();
}

template <typename E, int N, int ROWS>
int step_rows(const SsmParams& p, cudaStream_t st)
{
    const long long items = static_cast<long long>((p.B + ROWS - 1) / ROWS) * (p.D / 4) * (N / 4);
    ssm_step_kernel<E, N, ROWS><<<static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
    return launched();
}

// Two sequences a thread once the SMs are full of threads all the same (512 x 1024 channels of 64 states: 45.3 us, by one
// 47.2, by four 48.0).
template <typename E, int N>
int step(const SsmParams& p, cudaStream_t st)
{
    return static_cast<long long>(p.B) * p.D * (N / 16) >= 2LL * kSms * 1024 ? step_rows<E, N, 2>(p, st) : step_rows<E, N, 1>(p, st);
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
    const Split plan = plan_of(B, T, D, N, G);
    return std::max<size_t>(256, round256(static_cast<size_t>(plan.segments) * (B - plan.whole) * D * (N + 1) * 4));
}

int ssm_launch(int dtype, SsmParams& p, void* workspace, cudaStream_t st)
{
    const Split plan = plan_of(p.B, p.T, p.D, p.N, p.G);
    p.whole = plan.whole, p.segments = plan.segments, p.seg_len = plan.seg_len;
    p.seg_state = static_cast<float*>(workspace);
    p.seg_dt = p.seg_state + static_cast<size_t>(plan.segments) * (p.B - plan.whole) * p.D * p.N;
    return by_type(false, dtype, p, st);
}

int ssm_step_launch(int dtype, const SsmParams& p, cudaStream_t st) { return by_type(true, dtype, p, st); }

}  // namespace srwm
