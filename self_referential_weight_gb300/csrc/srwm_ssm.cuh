// srwm_ssm.cuh -- what the selective scan's kernels share: the step's softplus
// and the decays, a CTA's place and how the axis is cut, and the layout of the
// gradients' and the single token's lanes.
//
// There a lane holds four states of each of four channels, and the N / 4 lanes of
// a channel quad follow each other, so a warp holds 128 / (N / 4) channels.  A
// token's step and input come as one 16-byte load for four channels, B and C for
// four states, and a sum over states leaves through three or more shuffles for
// all four channels.  (The prompt's kernel, which has one such sum and not three,
// takes eight states of two channels: one shuffle.)
#pragma once

#include "srwm_ssm.h"
#include "srwm_vec.cuh"

namespace srwm {
namespace ssm {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 2;
constexpr int kThreads = 32 * kWarps;

template <int N>
struct Lay {
    static constexpr int kLanes = N / 4;              // of a channel quad
    static constexpr int kWarpCh = 4 * 32 / kLanes;   // channels of a warp
    static constexpr int kCh = kWarps * kWarpCh;      // of a CTA
};

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float2 ex2_2(float2 v) { return make_float2(ex2(v.x), ex2(v.y)); }

// A token's decays 2^(d A).  The approximate exponential's results near 1 lie below the value by 0.5e-8 to 2.9e-8 of it on
// average (measured for arguments from -0.3 to -1e-5), which a state that lasts for hundreds of tokens adds up; an argument
// larger by 2e-8 centres them (64 x 1024 tokens, dL/dA: 1.8e-6 -> 0.8e-6 of itself off).  A step of 0 still gives exactly 1.
// Results of positive arguments lie above the value by 0.3e-8 to 2e-8 (measured up to 1; 3.4e-8 at 16), so growth gets up
// to 3.4e-8 a token too much, half a rounding.
__device__ __forceinline__ float2 decay2(float2 d, float2 A) { return ex2_2(fma2(d, A, both(2.0e-8f))); }

// The smaller value, or NaN where one is.
__device__ __forceinline__ float2 min2(float2 v, float most)
{
    float2 r;
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r.x) : "f"(v.x), "f"(most));
    asm("min.NaN.f32 %0, %1, %2;" : "=f"(r.y) : "f"(v.y), "f"(most));
    return r;
}

// What a segment leaves of the state (or gradient) v that comes to it, and its own: 2^(A sum) v + own.  In two halves, each
// finite: growth past fp32's range keeps a state of 0 at 0, as it does token by token.
__device__ __forceinline__ float2 past_segment(float2 sum, float2 A, float2 v, float2 own)
{
    const float2 half = ex2_2(min2(mul2(mul2(sum, both(0.5f)), A), 126.f));
    return fma2(half, mul2(half, v), own);
}

// A step in units of log 2, log2(1 + 2^v) of its argument in these units: max(v, 0) + log2(1 + e), e = 2^-|v| in (0, 1].
// log(1 + e) = 2 artanh(e / (2 + e)), and artanh(s) / s is a polynomial in s^2 <= 1/9 (by Remez' exchange over that range,
// its constant term exact: up to 8.0e-9 of itself too small, 2.1e-8 with the coefficients rounded to fp32), here in
// w = (2 s)^2 and times log2 e.  Far negative arguments keep the relative
// precision that their own rounding leaves.  NaN gives NaN.
__device__ __forceinline__ float2 softplus2(float2 v)
{
    const float2 e = make_float2(ex2(-fabsf(v.x)), ex2(-fabsf(v.y)));
    const float2 d = fma2(e, both(0.5f), both(1.f));
    const float2 s = mul2(e, make_float2(rcp_approx(d.x), rcp_approx(d.y))), w = mul2(s, s);
    float2 r = fma2(w, both(7.9437119647e-04f), both(3.1511238925e-03f));
    r = fma2(r, w, both(1.8045010607e-02f));
    r = fma2(r, w, both(1.2022394380e-01f));
    r = fma2(r, w, both(1.4426950409e+00f));
    return fma2(s, r, make_float2(fmaxf(v.x, 0.f), fmaxf(v.y, 0.f)));
}

// z sigmoid(z), twice.
__device__ __forceinline__ float2 silu(float2 z)
{
    const float2 e = add2(ex2_2(mul2(z, both(-kLog2e))), both(1.f));
    return mul2(z, make_float2(rcp_approx(e.x), rcp_approx(e.y)));
}

// Four values, one per channel, summed over a quad's LANES lanes: every lane gets one channel's, quad_channel's.
template <int LANES>
__device__ __forceinline__ float quad_sum(float v0, float v1, float v2, float v3)
{
    const bool up = threadIdx.x & (LANES / 2), odd = threadIdx.x & (LANES / 4);
    const float a = (up ? v2 : v0) + __shfl_xor_sync(0xffffffffu, up ? v0 : v2, LANES / 2);
    const float b = (up ? v3 : v1) + __shfl_xor_sync(0xffffffffu, up ? v1 : v3, LANES / 2);
    float r = (odd ? b : a) + __shfl_xor_sync(0xffffffffu, odd ? a : b, LANES / 4);
#pragma unroll
    for (int o = LANES / 8; o > 0; o >>= 1) r += __shfl_xor_sync(0xffffffffu, r, o);
    return r;
}
template <int LANES>
__device__ __forceinline__ int quad_channel() { return (threadIdx.x & (LANES / 2) ? 2 : 0) + (threadIdx.x & (LANES / 4) ? 1 : 0); }
// One of the lanes that hold a channel's sum.
template <int LANES>
__device__ __forceinline__ bool quad_leader() { return (threadIdx.x & (LANES / 4 - 1)) == 0; }

__device__ __forceinline__ int valid_tokens(const int* lengths, int b, int T)
{
    return lengths ? min(max(__ldg(lengths + b), 0), T) : T;
}

// A CTA's place: a sequence, or a segment of one, and a range of a group's channels.
struct Place {
    int b, group, first, count;   // channels first .. first + count - 1 of D
    int segment, seg_len;
};
template <int CH>
__device__ __forceinline__ Place place_of(const SsmParams& p)
{
    const int dg = p.D / p.G, tiles = (dg + CH - 1) / CH;
    const unsigned i = blockIdx.x + p.first, range = i % (p.G * tiles), row = i / (p.G * tiles), split = row - p.whole;
    Place w;
    const bool whole = row < static_cast<unsigned>(p.whole);
    w.b = static_cast<int>(whole ? row : p.whole + split % (p.B - p.whole));
    w.segment = static_cast<int>(whole ? 0 : split / (p.B - p.whole));
    w.seg_len = whole ? max(p.T, 1) : p.seg_len;
    w.group = static_cast<int>(range) / tiles;
    const int tile = static_cast<int>(range) % tiles;
    w.first = w.group * dg + tile * CH;
    w.count = min(CH, dg - tile * CH);
    return w;
}
// Where segment j of the place's sequence has its channels in the segments' arrays, [segments, B - whole, D].
__device__ __forceinline__ size_t segment_at(const SsmParams& p, const Place& w, int j)
{
    return (static_cast<size_t>(j) * (p.B - p.whole) + (w.b - p.whole)) * p.D + w.first;
}

// Which sequences run whole and how the others are cut, for a kernel of `ctas` CTAs a sequence of which `slots` run at once.
// Waves of whole sequences fill the GPU; what is left over is cut into segments, up to `fill` CTAs of them, where it is less
// than `share` of a wave: a CTA by itself takes a large part of a full wave's time, the cut some more work.
struct Split {
    int whole, segments, seg_len;
};
inline Split split_of(long long B, long long ctas, int T, int slots, int fill, double share, int unit, int least)
{
    const Split uncut{static_cast<int>(B), 1, T > 0 ? T : 1};
    const long long whole = B * ctas / slots * slots / ctas, rest = (B - whole) * ctas;
    if (rest == 0 || rest > share * slots) return uncut;
    long long segments = fill / rest;
    if (segments > T / least) segments = T / least;
    if (segments > 64) segments = 64;
    if (segments < 2) return uncut;
    const int units = (T + unit - 1) / unit, per = static_cast<int>((units + segments - 1) / segments);
    return {static_cast<int>(whole), (units + per - 1) / per, per * unit};
}

// Four states of each of four channels, [.., D, N] from channel c and state n on: pairs are of channels.
__device__ __forceinline__ void load_states(const float* from, int N, bool on, float2 (&h)[2][4])
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        const float4 zero = make_float4(0.f, 0.f, 0.f, 0.f);
        const float4 a = on ? *reinterpret_cast<const float4*>(from + (2 * k) * N) : zero;
        const float4 b = on ? *reinterpret_cast<const float4*>(from + (2 * k + 1) * N) : zero;
        h[k][0] = make_float2(a.x, b.x), h[k][1] = make_float2(a.y, b.y);
        h[k][2] = make_float2(a.z, b.z), h[k][3] = make_float2(a.w, b.w);
    }
}
__device__ __forceinline__ void store_states(float* to, int N, const float2 (&h)[2][4])
{
#pragma unroll
    for (int k = 0; k < 2; ++k) {
        *reinterpret_cast<float4*>(to + (2 * k) * N) = make_float4(h[k][0].x, h[k][1].x, h[k][2].x, h[k][3].x);
        *reinterpret_cast<float4*>(to + (2 * k + 1) * N) = make_float4(h[k][0].y, h[k][1].y, h[k][2].y, h[k][3].y);
    }
}

}  // namespace ssm
}  // namespace srwm
