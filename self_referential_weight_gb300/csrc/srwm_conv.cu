// srwm_conv.cu -- the short causal convolution of each channel over its last W
// tokens, with an activation, and its gradients.
//
//   p_t = bias + sum_j w_j x_{t-W+1+j},   y_t = act(p_t)
//   g_t = dy_t act'(p_t),   dx_t = sum_j w_j g_{t+W-1-j},
//   dw_j = sum g_t x_{t-W+1+j},   dbias = sum g_t
// Memory bounds it: x (and dy) is to be read once and y (dx) written once.  A
// thread takes one vector of channels over a run of tokens, with the last W - 1
// inputs, the weights and the gradients' partial sums in registers.  Its rows
// come by asynchronous copies into a ring of its own in shared memory, so what is
// in flight takes no registers and no barrier; a run begins by reading the W - 1
// rows in front of it again, from L2.  64 x 1024 x 1024 in bf16 with W = 4 and SiLU
// take 49.3 us, 5.5 TB/s (with loads into registers 63); gradients of 512 x 512 x 256
// in fp32 134 us, 6.0 TB/s.
// Inputs before the first token, and the state that goes out, are rows of the
// state: row i of it stands W - 1 - i tokens before token 0, or before the
// sequence's end.
#include <cuda_runtime.h>

#include <algorithm>

#include "srwm.h"
#include "srwm_check.h"
#include "srwm_conv.h"
#include "srwm_sum.h"
#include "srwm_vec.cuh"

namespace srwm {
namespace {

constexpr int kSms = 152;
constexpr int kThreads = 128;
constexpr int kGroup = 4;         // tokens whose copies are waited for together
constexpr int kGroups = 4;        // groups of a thread's ring, all but one of them in flight
constexpr int kGradGroups = 3;
constexpr int kGradParts = 608;   // CTAs that take turns on the gradients' runs: four on each SM

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

// Tokens of a thread's run: as long as keeps the SMs full, since each begins with an empty ring and rows read again (the
// prompt above by 1024 threads an SM 49, by 512 54; 226 sequences of 31 x 16 in runs of 8 5.1 us, of 32 8.7).
int run_of(int B, int T, int vecs, int most, int threads)
{
    int run = 8;
    while (run < most && static_cast<long long>(B) * vecs * ((T + 2 * run - 1) / (2 * run)) >= kSms * threads) run *= 2;
    return run;
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

// The window moves on by one token: with several tokens unrolled these are other registers' names.
template <int W, int V>
__device__ __forceinline__ void shift(float (&win)[W][V])
{
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
        for (int k = 0; k < V; ++k) win[j][k] = win[j + 1][k];
}

template <typename E, int W, int ACT>
__global__ void __launch_bounds__(kThreads, 4) conv_kernel(const ConvParams p, int run_len, int runs)
{
    constexpr int V = vec<E>;
    extern __shared__ __align__(16) uint4 ring[];   // [groups][tokens][threads]: a thread's own rows on their way
    const int nv = p.D / V;
    const long long item = static_cast<long long>(blockIdx.x) * kThreads + threadIdx.x;
    const int c = static_cast<int>(item % nv) * V;
    const long long br = item / nv;
    const int run = static_cast<int>(br % runs);
    if (br / runs >= p.B) return;
    const int b = static_cast<int>(br / runs);
    const int n = valid_tokens(p.lengths, b, p.T);
    const int t0 = run * run_len, t1 = min(p.T, t0 + run_len), live = min(t1, n);
    const E* const x = static_cast<const E*>(p.x) + static_cast<size_t>(b) * p.T * p.ld + c;
    const size_t states = static_cast<size_t>(b) * (W - 1) * p.D + c;
    E* const y = static_cast<E*>(p.y) + static_cast<size_t>(b) * p.T * p.D + c;
    const uint4 zero = make_uint4(0, 0, 0, 0);
    // row i of the state or, past it, of the tokens
    auto row = [&](int i) {
        return i >= W - 1 ? load_vec<E>(x, static_cast<size_t>(i - (W - 1)) * p.ld)
               : p.state_in ? load_vec<E>(p.state_in, states + static_cast<size_t>(i) * p.D) : zero;
    };
    auto copy = [&](int group) {
#pragma unroll
        for (int a = 0; a < kGroup; ++a) {
            const int t = t0 + group * kGroup + a;
            if (t < live) cp_async16(smem_u32(ring + (group % kGroups * kGroup + a) * kThreads + threadIdx.x), x + static_cast<long long>(t) * p.ld, true);
        }
        cp_async_commit();
    };
    if (t0 < live) {
#pragma unroll
        for (int g = 0; g < kGroups - 1; ++g) copy(g);
        float w[W][V], bias[V], win[W][V];
        uint4 raw[W - 1];
#pragma unroll
        for (int i = 0; i < W - 1; ++i) raw[i] = row(t0 + i);
        load_weights<W, V>(p, c, w);
        load_bias<V>(p, c, bias);
#pragma unroll
        for (int i = 0; i < W - 1; ++i) unpack(raw[i], win[i], E{});
        auto token = [&](int t, const uint4& v) {
            unpack(v, win[W - 1], E{});
            float out[V];
#pragma unroll
            for (int k = 0; k < V; ++k) {
                out[k] = bias[k];
#pragma unroll
                for (int j = 0; j < W; ++j) out[k] = fmaf(w[j][k], win[j][k], out[k]);
                out[k] = conv_act<ACT>(out[k]);
            }
            store_vec<E>(y, static_cast<size_t>(t) * p.D, pack(out, E{}));
            shift(win);
        };
        for (int g = 0, t = t0; t < live; ++g, t += kGroup) {
            copy(g + kGroups - 1);
            cp_async_wait<kGroups - 1>();
            const uint4* const at = ring + g % kGroups * kGroup * kThreads + threadIdx.x;
            if (t + kGroup <= live) {
#pragma unroll
                for (int a = 0; a < kGroup; ++a) token(t + a, at[a * kThreads]);
            } else {
#pragma unroll 1
                for (int a = 0; t + a < live; ++a) token(t + a, at[a * kThreads]);
            }
        }
    }
    for (int t = max(t0, live); t < t1; ++t) store_vec<E>(y, static_cast<size_t>(t) * p.D, zero);
    if (p.state_out && run == (n > 0 ? (n - 1) / run_len : 0))   // the sequence ends here: its last rows, as they came
#pragma unroll
        for (int i = 0; i < W - 1; ++i) store_vec<E>(p.state_out, states + static_cast<size_t>(i) * p.D, row(n + i));
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
    int groups, vecs, slots, parts, run_len, runs;
};

GradPlan grad_plan(int B, int T, int D)
{
    GradPlan g{};
    const int nv = D / 4;
    g.vecs = std::min(nv, 32);
    g.groups = (nv + 31) / 32;
    g.slots = kThreads / g.vecs;
    g.run_len = run_of(B, T, nv, 256, 2048);
    g.runs = std::max(1, (T + g.run_len - 1) / g.run_len);
    const long long items = static_cast<long long>(B) * g.runs;
    g.parts = static_cast<int>(std::max(1LL, std::min<long long>((items + g.slots - 1) / g.slots, std::max(1, kGradParts / g.groups))));
    return g;
}

// dx (and dL/dstate_in) of every token, and a CTA's part of the parameters' gradients: part [parts, D W + D].
// At time t the inputs of rows t .. t + W - 1 (row i is token i - W + 1) get w_j g_t; row t is complete then.
template <typename E, int W, int ACT>
__global__ void __launch_bounds__(kThreads, 4) conv_grad_kernel(const ConvParams p, const GradPlan g)
{
    constexpr int V = 4;
    using Q = typename Quad<E>::type;
    extern __shared__ __align__(16) unsigned char ring_bytes[];
    Q* const ring = reinterpret_cast<Q*>(ring_bytes) + threadIdx.x;   // [groups][tokens][x | dy][threads]: a thread's own rows
    float (*const sums)[V] = reinterpret_cast<float (*)[V]>(ring_bytes);   // at the end, when no copy is on its way
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
        const int b = static_cast<int>(item % p.B), run = static_cast<int>(item / p.B);   // a thread's runs begin at different tokens: of uneven sequences the later ones are short
        const int n = valid_tokens(p.lengths, b, p.T);
        const int t0 = run * g.run_len, t1 = min(p.T, t0 + g.run_len);
        const E* const x = static_cast<const E*>(p.x) + static_cast<size_t>(b) * p.T * p.ld + c;
        const E* const dy = static_cast<const E*>(p.dy) + static_cast<size_t>(b) * p.T * p.D + c;
        E* const dx = static_cast<E*>(p.dx) + static_cast<size_t>(b) * p.T * p.ld_grad + c;
        const size_t states = static_cast<size_t>(b) * (W - 1) * p.D + c;
        const float none[V] = {};
        int t = t0;
        if (t0 < n || run == 0) {
            const int inner = min(t1, n), reach = min(t1 + W - 1, n);   // own tokens, and those that reach back to them
            auto copy = [&](int group) {
#pragma unroll
                for (int a = 0; a < kGroup; ++a) {
                    const int i = t0 + group * kGroup + a;
                    if (i < reach) {
                        Q* const to = ring + (group % kGradGroups * kGroup + a) * 2 * kThreads;
                        cp_async_own<sizeof(Q)>(smem_u32(to), x + static_cast<long long>(i) * p.ld);
                        cp_async_own<sizeof(Q)>(smem_u32(to + kThreads), dy + static_cast<long long>(i) * p.D);
                    }
                }
                cp_async_commit();
            };
#pragma unroll
            for (int q = 0; q < kGradGroups - 1; ++q) copy(q);
            float win[W][V], acc[W][V];   // inputs of rows t .. t + W - 1; their gradients so far
#pragma unroll
            for (int i = 0; i < W; ++i)
#pragma unroll
                for (int k = 0; k < V; ++k) win[i][k] = acc[i][k] = 0.f;
#pragma unroll
            for (int i = 0; i < W - 1; ++i) {
                const int from = t0 - (W - 1) + i;
                if (from >= 0)
                    unpack_quad(load_quad<E>(x, static_cast<size_t>(from) * p.ld), win[i], E{});
                else if (p.state_in)
                    unpack_quad(load_quad<E>(p.state_in, states + static_cast<size_t>(t0 + i) * p.D), win[i], E{});
            }
            // the gradient of a valid token's sum reaches its inputs and, for the run's own tokens, the parameters
            auto token = [&](const Q& rx, const Q& rd, bool mine) {
                float d[V];
                unpack_quad(rx, win[W - 1], E{});
                unpack_quad(rd, d, E{});
#pragma unroll
                for (int k = 0; k < V; ++k) {
                    float v = bias[k];
#pragma unroll
                    for (int j = 0; j < W; ++j) v = fmaf(w[j][k], win[j][k], v);
                    const float gr = d[k] * conv_slope<ACT>(v);
#pragma unroll
                    for (int j = 0; j < W; ++j) acc[j][k] = j < W - 1 ? fmaf(w[j][k], gr, acc[j][k]) : w[j][k] * gr;
                    if (mine) {
                        db[k] += gr;
#pragma unroll
                        for (int j = 0; j < W; ++j) dw[j][k] = fmaf(gr, win[j][k], dw[j][k]);
                    }
                }
            };
            // row `now` is complete: a token's dx, or a row of the state that came in
            auto emit = [&](int now) {
                const int at = now - (W - 1);
                if (at >= t0)
                    store_quad<E>(dx, static_cast<size_t>(at) * p.ld_grad, pack_quad(acc[0], E{}));
                else if (at < 0 && p.state_out)
                    store_quad<E>(p.state_out, states + static_cast<size_t>(now) * p.D, pack_quad(acc[0], E{}));
                shift(acc);
                shift(win);
            };
            for (int q = 0; t < reach; ++q, t += kGroup) {
                copy(q + kGradGroups - 1);
                cp_async_wait<kGradGroups - 1>();
                const Q* const at = ring + q % kGradGroups * kGroup * 2 * kThreads;
                if (t + kGroup <= inner) {
#pragma unroll
                    for (int a = 0; a < kGroup; ++a) {
                        token(at[a * 2 * kThreads], at[(a * 2 + 1) * kThreads], true);
                        emit(t + a);
                    }
                } else {
#pragma unroll 1
                    for (int a = 0; a < kGroup && t + a < reach; ++a) {
                        token(at[a * 2 * kThreads], at[(a * 2 + 1) * kThreads], t + a < t1);
                        emit(t + a);
                    }
                }
            }
            // the rows behind the sequence's end belong to the state that went out
            for (t = reach; t < inner + W - 1; ++t) {
#pragma unroll
                for (int k = 0; k < V; ++k) acc[W - 1][k] = 0.f;
                if (p.dstate) {
                    float d[V];
                    unpack_quad(load_quad<E>(p.dstate, states + static_cast<size_t>(t - n) * p.D), d, E{});
#pragma unroll
                    for (int k = 0; k < V; ++k) acc[0][k] += d[k];
                }
                emit(t);
            }
            t = inner;   // dx is written up to here
        }
        for (t = max(t, t0); t < t1; ++t) store_quad<E>(dx, static_cast<size_t>(t) * p.ld_grad, pack_quad(none, E{}));
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
        for (int i = threadIdx.x; i < g.vecs * V; i += kThreads) {
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
    const int run = run_of(p.B, p.T, p.D / vec<E>, 256, 1024), runs = std::max(1, (p.T + run - 1) / run);
    const long long items = static_cast<long long>(p.D / vec<E>) * runs * p.B;
    constexpr int smem = kGroups * kGroup * kThreads * 16;
    conv_kernel<E, W, ACT><<<static_cast<unsigned>((items + kThreads - 1) / kThreads), kThreads, smem, st>>>(p, run, runs);
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
    constexpr int smem = kGradGroups * kGroup * 2 * kThreads * static_cast<int>(sizeof(typename Quad<E>::type));
    conv_grad_kernel<E, W, ACT><<<static_cast<unsigned>(g.groups) * g.parts, kThreads, smem, st>>>(p, g);
    const int rc = launched();
    if (rc != SRWM_OK || !params) return rc;
    return sum_launch({p.part, g.parts, {p.dweight, p.dbias, nullptr}, {static_cast<long long>(p.D) * W, p.D, 0}, false}, st);
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
