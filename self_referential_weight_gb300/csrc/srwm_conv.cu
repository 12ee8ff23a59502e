// srwm_conv.cu -- the short causal convolution of each channel over its last W
// tokens, with an activation, and its gradients.
//
//   p_t = bias + sum_j w_j x_{t-W+1+j},   y_t = act(p_t)
//   g_t = dy_t act'(p_t),   dx_t = sum_j w_j g_{t+W-1-j},
//   dw_j = sum g_t x_{t-W+1+j},   dbias = sum g_t
// Memory bounds it: x (and dy) is to be read once and y (dx) written once.  A
// thread takes one vector of channels over a run of tokens, with the last W - 1
// inputs, the weights and the gradients' partial sums in registers, and several
// tokens' loads in flight; a run begins by reading the W - 1 rows in front of it
// again, from L2.  Inputs before the first token, and the state that goes out,
// are rows of the state: row i of it stands W - 1 - i tokens before token 0, or
// before the sequence's end.
#include <cuda_runtime.h>

#include <algorithm>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_conv.h"
#include "srwm_sum.h"
#include "srwm_vec.cuh"

namespace srwm {
namespace {

constexpr int kThreads = 128;
constexpr int kRun = 32;          // tokens of a thread's run
constexpr int kAhead = 8;         // of which are loaded at once
constexpr int kGradThreads = 256;
constexpr int kGradParts = 608;   // partial sums of a channel's parameters: four CTAs on each SM

template <int ACT>
__device__ __forceinline__ float conv_act(float v) { return ACT == SRWM_ACT_SILU ? v * sigmoid(v) : v; }

template <int ACT>
__device__ __forceinline__ float conv_slope(float v)
{
    if constexpr (ACT == SRWM_ACT_SILU) {
        const float e = sigmoid(v);
        return e * fmaf(v, 1.f - e, 1.f);
    }
    return 1.f;
}

__device__ __forceinline__ int valid_tokens(const int* lengths, int b, int T)
{
    return lengths ? min(max(__ldg(lengths + b), 0), T) : T;
}

template <int W, int V>
__device__ __forceinline__ void load_weights(const ConvParams& p, int c, float (&w)[W][V])
{
    float flat[V * W];
#pragma unroll
    for (int i = 0; i < V * W; i += 4) {
        const float4 q = __ldg(reinterpret_cast<const float4*>(p.weight + static_cast<size_t>(c) * W + i));
        flat[i] = q.x, flat[i + 1] = q.y, flat[i + 2] = q.z, flat[i + 3] = q.w;
    }
#pragma unroll
    for (int j = 0; j < W; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) w[j][k] = flat[k * W + j];
}

template <int V>
__device__ __forceinline__ void load_bias(const ConvParams& p, int c, float (&bias)[V])
{
#pragma unroll
    for (int k = 0; k < V; k += 4) {
        const float4 q = p.bias ? __ldg(reinterpret_cast<const float4*>(p.bias + c + k)) : make_float4(0.f, 0.f, 0.f, 0.f);
        bias[k] = q.x, bias[k + 1] = q.y, bias[k + 2] = q.z, bias[k + 3] = q.w;
    }
}

template <typename E, int W, int ACT>
__global__ void __launch_bounds__(kThreads) conv_kernel(const ConvParams p, int runs)
{
    constexpr int V = vec<E>;
    const int nv = p.D / V;
    const long long item = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const int c = static_cast<int>(item % nv) * V;
    const long long br = item / nv;
    const int run = static_cast<int>(br % runs);
    if (br / runs >= p.B) return;
    const int b = static_cast<int>(br / runs);
    const int n = valid_tokens(p.lengths, b, p.T);
    const int t0 = run * kRun, t1 = min(p.T, t0 + kRun), live = min(t1, n);
    const E* const x = static_cast<const E*>(p.x) + static_cast<size_t>(b) * p.T * p.ld + c;
    const size_t states = static_cast<size_t>(b) * (W - 1) * p.D + c;
    E* const y = static_cast<E*>(p.y) + static_cast<size_t>(b) * p.T * p.D + c;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    const bool last = run == (n > 0 ? (n - 1) / kRun : 0);
    int t = t0;
    if (t0 < live || last) {
        float w[W][V], bias[V], win[W][V];
        load_weights<W, V>(p, c, w);
        load_bias<V>(p, c, bias);
        uint4 old[W - 1];   // rows as they came: the state that goes out is not rounded again
#pragma unroll
        for (int i = 0; i < W - 1; ++i) {
            const int from = t0 - (W - 1) + i;
            old[i] = from >= 0 ? load_vec<E>(x, static_cast<size_t>(from) * p.ld)
                     : p.state_in ? load_vec<E>(p.state_in, states + static_cast<size_t>(t0 + i) * p.D) : zero;
            unpack(old[i], win[i], E{});
        }
        while (t < live) {
            uint4 raw[kAhead];
#pragma unroll
            for (int a = 0; a < kAhead; ++a)
                if (t + a < live) raw[a] = load_vec<E>(x, static_cast<size_t>(t + a) * p.ld);
#pragma unroll
            for (int a = 0; a < kAhead; ++a) {
                if (t + a >= live) break;
                unpack(raw[a], win[W - 1], E{});
                float out[V];
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float v = bias[k];
#pragma unroll
                    for (int j = 0; j < W; ++j) v = fmaf(w[j][k], win[j][k], v);
                    out[k] = conv_act<ACT>(v);
                }
                store_vec<E>(y, static_cast<size_t>(t + a) * p.D, pack(out, E{}));
#pragma unroll
                for (int j = 0; j < W - 1; ++j) {
                    old[j] = j < W - 2 ? old[j + 1] : raw[a];
#pragma unroll
                    for (int k = 0; k < V; ++k) win[j][k] = win[j + 1][k];
                }
            }
            t = min(t + kAhead, live);
        }
        if (last && p.state_out) {
#pragma unroll
            for (int i = 0; i < W - 1; ++i) store_vec<E>(p.state_out, states + static_cast<size_t>(i) * p.D, old[i]);
        }
    }
    for (t = max(t0, live); t < t1; ++t) store_vec<E>(y, static_cast<size_t>(t) * p.D, zero);
}

template <typename E, int W, int ACT>
__global__ void __launch_bounds__(kThreads) conv_step_kernel(const ConvParams p)
{
    constexpr int V = vec<E>;
    const int nv = p.D / V;
    const long long item = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const int c = static_cast<int>(item % nv) * V;
    const long long b = item / nv;
    if (b >= p.B) return;
    const size_t states = static_cast<size_t>(b) * (W - 1) * p.D + c;
    uint4 row[W];
#pragma unroll
    for (int i = 0; i < W - 1; ++i)
        row[i] = *reinterpret_cast<const uint4*>(static_cast<const E*>(p.state_in) + states + static_cast<size_t>(i) * p.D);
    row[W - 1] = load_vec<E>(p.x, static_cast<size_t>(b) * p.ld + c);
    float w[W][V], out[V];
    load_weights<W, V>(p, c, w);
    load_bias<V>(p, c, out);
#pragma unroll
    for (int j = 0; j < W; ++j) {
        float v[V];
        unpack(row[j], v, E{});
#pragma unroll
        for (int k = 0; k < V; ++k) out[k] = fmaf(w[j][k], v[k], out[k]);
    }
#pragma unroll
    for (int k = 0; k < V; ++k) out[k] = conv_act<ACT>(out[k]);
    store_vec<E>(p.y, static_cast<size_t>(b) * p.D + c, pack(out, E{}));
#pragma unroll
    for (int i = 0; i < W - 1; ++i) store_vec<E>(p.state_out, states + static_cast<size_t>(i) * p.D, row[i + 1]);
}

// How the threads of conv_grad_kernel share the channels: groups of up to 32 vectors of four channels, a run per slot.
struct GradPlan {
    int groups, vecs, slots, parts, runs;
};

GradPlan grad_plan(int B, int T, int D)
{
    GradPlan g{};
    const int nv = D / 4;
    g.vecs = std::min(nv, 32);
    g.groups = (nv + 31) / 32;
    g.slots = kGradThreads / g.vecs;
    g.runs = std::max(1, (T + kRun - 1) / kRun);
    const long long items = static_cast<long long>(B) * g.runs;
    g.parts = static_cast<int>(std::max(1LL, std::min<long long>((items + g.slots - 1) / g.slots, std::max(1, kGradParts / g.groups))));
    return g;
}

// dx (and dL/dstate_in) of every token, and a CTA's part of the parameters' gradients: part [parts, D W + D].
// At time t the inputs of rows t .. t + W - 1 (row i is token i - W + 1) get w_j g_t; row t is complete then.
template <typename E, int W, int ACT>
__global__ void __launch_bounds__(kGradThreads) conv_grad_kernel(const ConvParams p, const GradPlan g)
{
    constexpr int V = 4, U = 4;
    using Q = typename Quad<E>::type;
    __shared__ float sums[kGradThreads][V];
    const int group = blockIdx.x % g.groups, part = blockIdx.x / g.groups;
    const int lane = threadIdx.x % g.vecs, slot = threadIdx.x / g.vecs;
    const int c = (group * 32 + lane) * V;
    const bool on = slot < g.slots && c < p.D;
    float w[W][V], bias[V], dw[W][V], db[V];
#pragma unroll
    for (int k = 0; k < V; ++k) {
        db[k] = 0.f;
#pragma unroll
        for (int j = 0; j < W; ++j) dw[j][k] = 0.f;
    }
    const long long items = on ? static_cast<long long>(p.B) * g.runs : 0;
    if (on) {
        load_weights<W, V>(p, c, w);
        load_bias<V>(p, c, bias);
    }
    for (long long item = static_cast<long long>(part) * g.slots + slot; item < items; item += static_cast<long long>(g.parts) * g.slots) {
        const int b = static_cast<int>(item / g.runs), run = static_cast<int>(item % g.runs);
        const int n = valid_tokens(p.lengths, b, p.T);
        const int t0 = run * kRun, t1 = min(p.T, t0 + kRun);
        const E* const x = static_cast<const E*>(p.x) + static_cast<size_t>(b) * p.T * p.ld + c;
        const E* const dy = static_cast<const E*>(p.dy) + static_cast<size_t>(b) * p.T * p.D + c;
        E* const dx = static_cast<E*>(p.dx) + static_cast<size_t>(b) * p.T * p.ld_grad + c;
        const size_t states = static_cast<size_t>(b) * (W - 1) * p.D + c;
        float win[W][V], acc[W][V];   // inputs of rows t .. t + W - 1; their gradients so far
#pragma unroll
        for (int i = 0; i < W; ++i)
#pragma unroll
            for (int k = 0; k < V; ++k) win[i][k] = acc[i][k] = 0.f;
        if (t0 < n)
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const int from = t0 - (W - 1) + i;
                if (from >= 0)
                    unpack_quad(load_quad<E>(x, static_cast<size_t>(from) * p.ld), win[i], E{});
                else if (p.state_in)
                    unpack_quad(load_quad<E>(p.state_in, states + static_cast<size_t>(t0 + i) * p.D), win[i], E{});
            }
        const int end = t1 + W - 1;
        for (int t = t0; t < end; t += U) {
            Q rx[U], rd[U];
#pragma unroll
            for (int a = 0; a < U; ++a)
                if (t + a < end && t + a < n) {
                    rx[a] = load_quad<E>(x, static_cast<size_t>(t + a) * p.ld);
                    rd[a] = load_quad<E>(dy, static_cast<size_t>(t + a) * p.D);
                }
#pragma unroll
            for (int a = 0; a < U; ++a) {
                const int now = t + a;
                if (now >= end) break;
                if (now < n) {
                    float d[V];
                    unpack_quad(rx[a], win[W - 1], E{});
                    unpack_quad(rd[a], d, E{});
                    const bool mine = now < t1;
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        float v = bias[k];
#pragma unroll
                        for (int j = 0; j < W; ++j) v = fmaf(w[j][k], win[j][k], v);
                        const float gr = d[k] * conv_slope<ACT>(v);
#pragma unroll
                        for (int j = 0; j < W; ++j) acc[j][k] = fmaf(w[j][k], gr, acc[j][k]);
                        if (mine) {
                            db[k] += gr;
#pragma unroll
                            for (int j = 0; j < W; ++j) dw[j][k] = fmaf(gr, win[j][k], dw[j][k]);
                        }
                    }
                }
                const int token = now - (W - 1);
                if (now >= n && token < n && p.dstate) {   // row `now` is row now - n of the state that went out
                    float d[V];
                    unpack_quad(load_quad<E>(p.dstate, states + static_cast<size_t>(now - n) * p.D), d, E{});
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[0][k] += d[k];
                }
                if (token >= t0) {
                    if (token >= n)
#pragma unroll
                        for (int k = 0; k < V; ++k) acc[0][k] = 0.f;
                    store_quad<E>(dx, static_cast<size_t>(token) * p.ld_grad, pack_quad(acc[0], E{}));
                } else if (token < 0 && run == 0 && p.state_out) {
                    store_quad<E>(p.state_out, states + static_cast<size_t>(now) * p.D, pack_quad(acc[0], E{}));
                }
#pragma unroll
                for (int j = 0; j < W; ++j)
#pragma unroll
                    for (int k = 0; k < V; ++k) {
                        acc[j][k] = j < W - 1 ? acc[j + 1][k] : 0.f;
                        if (j < W - 1) win[j][k] = win[j + 1][k];
                    }
            }
        }
    }
    griddep_launch();
    if (!p.part) return;
    float* const to = p.part + static_cast<size_t>(part) * p.D * (W + 1);
#pragma unroll
    for (int j = 0; j <= W; ++j) {   // the slots' sums in order, a column of the parameters at a time
        __syncthreads();
#pragma unroll
        for (int k = 0; k < V; ++k) sums[threadIdx.x][k] = j < W ? dw[j < W ? j : 0][k] : db[k];
        __syncthreads();
        for (int i = threadIdx.x; i < g.vecs * V; i += kGradThreads) {
            const int at = group * 32 * V + i;
            if (at >= p.D) continue;
            float a = 0.f;
            for (int s = 0; s < g.slots; ++s) a += sums[s * g.vecs + i / V][i % V];
            to[j < W ? static_cast<size_t>(at) * W + j : static_cast<size_t>(p.D) * W + at] = a;
        }
    }
}

template <typename E, int W, int ACT>
int forward(const ConvParams& p, cudaStream_t st)
{
    const int runs = std::max(1, (p.T + kRun - 1) / kRun);
    const long long items = static_cast<long long>(p.D / vec<E>) * runs * p.B;
    conv_kernel<E, W, ACT><<<static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, 0, st>>>(p, runs);
    return launched();
}

template <typename E, int W, int ACT>
int step(const ConvParams& p, cudaStream_t st)
{
    const long long items = static_cast<long long>(p.D / vec<E>) * p.B;
    conv_step_kernel<E, W, ACT><<<static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, 0, st>>>(p);
    return launched();
}

template <typename E, int W, int ACT>
int backward(const ConvParams& p0, cudaStream_t st)
{
    ConvParams p = p0;
    const GradPlan g = grad_plan(p.B, p.T, p.D);
    const bool params = p.dweight || p.dbias;
    if (!params) p.part = nullptr;
    conv_grad_kernel<E, W, ACT><<<static_cast<unsigned>(g.groups) * g.parts, kGradThreads, 0, st>>>(p, g);
    const int rc = launched();
    if (rc != SRWM_OK || !params) return rc;
    return sum_launch({p.part, g.parts, {p.dweight, p.dbias, nullptr}, {static_cast<long long>(p.D) * W, p.D, 0}}, st);
}

enum Way { kForward, kStep, kBackward };

template <typename E, int W, int ACT>
int by_way(Way way, const ConvParams& p, cudaStream_t st)
{
    return way == kForward ? forward<E, W, ACT>(p, st) : way == kStep ? step<E, W, ACT>(p, st) : backward<E, W, ACT>(p, st);
}

template <typename E, int W>
int by_act(Way way, int activation, const ConvParams& p, cudaStream_t st)
{
    return activation == SRWM_ACT_SILU ? by_way<E, W, SRWM_ACT_SILU>(way, p, st) : by_way<E, W, SRWM_ACT_NONE>(way, p, st);
}

template <typename E>
int by_width(Way way, int W, int activation, const ConvParams& p, cudaStream_t st)
{
    return W == 2 ? by_act<E, 2>(way, activation, p, st) : W == 3 ? by_act<E, 3>(way, activation, p, st) : by_act<E, 4>(way, activation, p, st);
}

int by_type(Way way, int dtype, int W, int activation, const ConvParams& p, cudaStream_t st)
{
    if (dtype == SRWM_F32) return by_width<float>(way, W, activation, p, st);
    if (dtype == SRWM_BF16) return by_width<__nv_bfloat16>(way, W, activation, p, st);
    return by_width<__half>(way, W, activation, p, st);
}

}  // namespace

size_t conv_backward_scratch(int B, int T, int D, int W)
{
    return round256(static_cast<size_t>(grad_plan(B, T, D).parts) * D * (W + 1) * 4);
}

int conv_launch(int dtype, int W, int activation, const ConvParams& p, cudaStream_t st) { return by_type(kForward, dtype, W, activation, p, st); }
int conv_step_launch(int dtype, int W, int activation, const ConvParams& p, cudaStream_t st) { return by_type(kStep, dtype, W, activation, p, st); }
int conv_backward_launch(int dtype, int W, int activation, const ConvParams& p, cudaStream_t st) { return by_type(kBackward, dtype, W, activation, p, st); }

}  // namespace srwm
