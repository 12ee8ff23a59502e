// srwm_linattn.cuh -- the chunked kernel of the primitive in srwm_linattn.h.
//
// One CTA runs one stream (sequence, head) of one role, or one segment of its
// length, in chunks of D tokens.  Per chunk (i, j positions in it, P = a b^T,
// g the decay):
//   out_i = alpha_o [ g^(i+1-delta) a_i X  +  alpha_u sum_{j<=i} g^(i-j) P_ij c_j ]
//   X     = g^n X + alpha_u sum_j g^(n-1-j+delta) b_j c_j^T
// (delta = 0 in order, 1 in reverse).  Half of the CTA's D / 8 warps work on
// each line, at the same time: the chunk's outputs need X before the chunk,
// and X's update needs nothing of the outputs.
//   State warp w holds rows 16w .. 16w + 15 of X in fp32 accumulators, and
// leaves an fp16 copy of X in shared memory after each chunk.
//   Output warp w computes output rows 16w .. 16w + 15: a X from that copy,
// then the column groups below the diagonal, where the decay is a product of a
// row's, a group's and a column's factor, then the diagonal 16 x 16 block.
// Blocks above the diagonal are not computed.
// Per token that is 2 D^2 multiply-adds by the state and about 1.25 D^2 inside
// the chunk, whatever T is; a warp's share of every matrix is a 16-row strip.
//
// The products run on the tensor cores in fp16 (mma.sync), with fp32 sums.
// mma.sync rather than tcgen05.mma at D = 16 and 32, whose strips would fill an
// eighth or a quarter of a 128-row product; D = 64 comes here where the axis is
// split, in fp16, and below 128 tokens (srwm_linattn_tc.cu takes the rest).  The
// shortest sequences run token by token (srwm_linattn_scan.cu).
// What bounds it is instruction issue: 2048 ragged streams of up to 512 tokens
// in bf16 at D = 32 (184 MB) take 55 us, 0.49 of the copy rate, with 59 % of
// the issue slots busy over the whole launch, its uneven end included.
//
// Range and precision.  Each group of 16 tokens of a, b and c is scaled by a
// power of two that puts its largest magnitude into [2^13, 2^14), exactly; all
// later factors carry exponents as integers and are normalised to the largest
// one in use, so fp16's range never matters.  fp32 values are split into a high
// and a low fp16 (22 bits); three of the four products are kept.  bf16 and
// fp16 values are one fp16 exactly.  The weighted rows of b always enter the
// state as pairs, so the state is good to fp32 for every type.  The score P
// and the state's copy enter their products as pairs for fp32 and fp16, and as
// one fp16 (2^-11 of each value) for bf16, whose outputs round by 2^-8: as pairs
// the batch above takes 64.6 us, for the same relative error but for 0.6 % of it.
#pragma once

#include <cuda_runtime.h>

#include <type_traits>

#include "srwm_elem.cuh"
#include "srwm_linattn.h"
#include "srwm_mma.cuh"
#include "srwm_ptx.cuh"

namespace srwm {

constexpr int kNoValue = -4000;   // exponent of a group of zeros

// 2^e, 0 below the normal range, 2^127 above.
__device__ __forceinline__ float pow2i(int e)
{
    return e < -126 ? 0.f : __int_as_float((min(e, 127) + 127) << 23);
}

// log2 of the decay per token: <= 0 and finite, so that multiples of it are; NaN stays NaN.
__device__ __forceinline__ float decay_log2(float log_decay)
{
    return isnan(log_decay) ? log_decay : fmaxf(fminf(log_decay, 0.f) * 1.4426950408889634f, -16384.f);
}

// g^n as X -> m X + c X: with c = 1 and m = g^n - 1 where g^n is near 1, so
// that a state kept over many chunks does not lose the bits of 1 - g^n.
struct Decay {
    float m, c;
};
__device__ __forceinline__ Decay decay_over(float lg2, int n)
{
    const float x = lg2 * static_cast<float>(n) * 0.6931471805599453f;
    return x > -0.5f ? Decay{expm1f(x), 1.f} : Decay{expf(x), 0.f};
}

template <typename E, int D>
struct LinTile {
    static constexpr int kWarps = D / 16;                                   // of either kind
    static constexpr int kThreads = 2 * 32 * kWarps;
    static constexpr int NI = sizeof(E) == 4 ? 2 : 1;                       // fp16 terms of an input
    static constexpr int NM = std::is_same<E, __nv_bfloat16>::value ? 1 : 2;  // of a score or the state's copy
    static constexpr int kStages = D == 64 ? 2 : 3;                         // chunks in shared memory
    static constexpr int kRow = 2 * D;                                      // bytes of a row of one term
    static constexpr int kGroup = 16 * D * static_cast<int>(sizeof(E));      // 16 tokens: raw, later their terms
    static constexpr int kTile = kWarps * kGroup;                           // D tokens
    static constexpr int kState = D * kRow;                                 // one term of the state's copy
    static constexpr int kSmem = kStages * 3 * kTile + NM * kState;
    static constexpr int kSmemState = kStages * 2 * kTile;                  // the state-only pass
    static constexpr int kPieces = kGroup / 512;                            // 16-byte pieces per lane and group
    static constexpr int kPerRow = D * static_cast<int>(sizeof(E)) / 16;    // pieces of a row
};

// 16-byte piece `c` of row r, placed so that eight consecutive rows' pieces of
// one column lie in distinct banks.
template <int D>
__device__ __forceinline__ int swizzle(int r, int c)
{
    if constexpr (D == 64) return c ^ (r & 7);
    if constexpr (D == 32) return c ^ ((r >> 1) & 3);
    return c ^ ((r >> 2) & 1);
}

// Address of piece c of term k of tile row r.
template <typename E, int D>
__device__ __forceinline__ uint32_t tile_at(uint32_t tile, int r, int c, int k = 0)
{
    using L = LinTile<E, D>;
    return tile + (r >> 4) * L::kGroup + k * 16 * L::kRow + (r & 15) * L::kRow + (swizzle<D>(r, c) << 4);
}

template <int D>
__device__ __forceinline__ uint32_t state_at(uint32_t base, int r, int c, int k)
{
    return base + k * D * 2 * D + r * 2 * D + (swizzle<D>(r, c) << 4);
}

// A warp's walk over its group's 16 rows of one tensor, chunk by chunk.
template <typename E, int D>
struct GroupLoader {
    using L = LinTile<E, D>;
    static constexpr int kRowStep = 32 / L::kPerRow;   // rows between a lane's pieces
    const char* base;       // the stream's first token
    const char* at;         // this lane's first piece in the next chunk
    long long row, chunk;   // bytes, with the direction's sign
    int pos;                // position of that piece's row

    __device__ __forceinline__ GroupLoader(const void* tensor, long long ld, long long token0, int column, int first,
                                           int n, bool reverse)
    {
        const int lane = threadIdx.x & 31;
        base = reinterpret_cast<const char*>(static_cast<const E*>(tensor) + token0 * ld + column) + lane % L::kPerRow * 16;
        row = ld * static_cast<long long>(sizeof(E)) * (reverse ? -1 : 1);
        chunk = row * D;
        pos = first + lane / L::kPerRow;
        at = base + (reverse ? -row * (n - 1) : 0) + row * pos;
    }
    // Starts the copy of the next chunk's rows; those at or past n are not read and become zeros.
    __device__ __forceinline__ void next(uint32_t group, int n)
    {
        const int lane = threadIdx.x & 31;
#pragma unroll
        for (int q = 0; q < L::kPieces; ++q) {
            const int p = lane + 32 * q, r = p / L::kPerRow, c = p % L::kPerRow;
            // 16-bit types land where their fp16 values will stay; fp32 rows lie plain until they are split
            const uint32_t dst = sizeof(E) == 2 ? group + r * L::kRow + (swizzle<D>(r, c) << 4) : group + p * 16;
            const bool ok = pos + q * kRowStep < n;
            cp_async16(dst, ok ? at + row * (q * kRowStep) : base, ok);
        }
        at += chunk;
        pos += D;
    }
};

__device__ __forceinline__ float2 pair_to_f(uint32_t v, __nv_bfloat16)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_to_f(uint32_t v, __half) { return unpack_half2(v); }

__device__ __forceinline__ uint32_t pack_pair(float x, float y, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_pair(float x, float y, __half) { return pack_half2(x, y); }

// Turns this warp's landed group into scaled fp16 terms in place.  Every lane
// converts the pieces it copied.  Returns the exponent e of the group: value = term * 2^e.
template <typename E, int D>
__device__ __forceinline__ int convert_group(uint32_t group)
{
    using L = LinTile<E, D>;
    const int lane = threadIdx.x & 31;
    constexpr int per_row = L::kPerRow;
    uint32_t v[L::kPieces][4];
    uint32_t at[L::kPieces];
    uint32_t top = 0;
#pragma unroll
    for (int q = 0; q < L::kPieces; ++q) {
        const int p = lane + 32 * q, r = p / per_row, c = p % per_row;
        at[q] = sizeof(E) == 2 ? group + r * L::kRow + (swizzle<D>(r, c) << 4) : group + p * 16;
        asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                     : "=r"(v[q][0]), "=r"(v[q][1]), "=r"(v[q][2]), "=r"(v[q][3])
                     : "r"(at[q]));
#pragma unroll
        for (int k = 0; k < 4; ++k) {
            // largest magnitude as bits (of fp32 or of both 16-bit halves): for
            // non-negative numbers the order of the bits is the order of the values
            if constexpr (sizeof(E) == 4)
                top = max(top, v[q][k] & 0x7fffffffu);
            else
                top = __vmaxu2(top, v[q][k] & 0x7fff7fffu);
        }
    }
    int e;
    if constexpr (sizeof(E) == 2) top = max(top & 0xffffu, top >> 16);
    top = __reduce_max_sync(0xffffffffu, top);
    if constexpr (std::is_same<E, __half>::value)
        top = __float_as_uint(__half2float(__ushort_as_half(static_cast<unsigned short>(top))));
    else if constexpr (sizeof(E) == 2)
        top <<= 16;
    const int ex = max(static_cast<int>(top >> 23), 14);   // 2^(ex-127) <= top < 2^(ex-126)
    e = top == 0 ? kNoValue : ex - 140;
    const float sc = __int_as_float((267 - ex) << 23);     // 2^(140 - ex): top * sc in [2^13, 2^14)
    if constexpr (sizeof(E) == 2) {
#pragma unroll
        for (int q = 0; q < L::kPieces; ++q) {
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const float2 f = mul2(pair_to_f(v[q][k], E{}), both(sc));
                v[q][k] = pack_half2(f.x, f.y);
            }
            asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(at[q]), "r"(v[q][0]), "r"(v[q][1]),
                         "r"(v[q][2]), "r"(v[q][3])
                         : "memory");
        }
    } else {
        __syncwarp();   // every lane has read its raw pieces; the terms go over them
#pragma unroll
        for (int q = 0; q < L::kPieces; ++q) {
            const int p = lane + 32 * q, r = p / per_row, c = p % per_row;
            uint32_t hi[2], lo[2];
            split_half2(__uint_as_float(v[q][0]) * sc, __uint_as_float(v[q][1]) * sc, hi[0], lo[0]);
            split_half2(__uint_as_float(v[q][2]) * sc, __uint_as_float(v[q][3]) * sc, hi[1], lo[1]);
            const uint32_t dst = group + r * L::kRow + (swizzle<D>(r, c >> 1) << 4) + (c & 1) * 8;
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(dst), "r"(hi[0]), "r"(hi[1]) : "memory");
            asm volatile("st.shared.v2.u32 [%0], {%1,%2};" ::"r"(dst + 16 * L::kRow), "r"(lo[0]), "r"(lo[1]) : "memory");
        }
    }
    return e;
}

__device__ __forceinline__ void named_arrive(int id, int threads)
{
    asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory");
}
__device__ __forceinline__ void named_sync(int id, int threads)
{
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

template <typename E, int D>
struct LinShared {
    int exp[LinTile<E, D>::kStages][2][LinTile<E, D>::kWarps];   // exponents of b's and c's groups
    int state_exp;                                               // of the state's copy
    float top[LinTile<E, D>::kWarps];
};

// What both kinds of warps know.
template <typename E, int D, bool STATE_ONLY>
struct LinWork {
    using L = LinTile<E, D>;
    const LinParams& p;
    const LinRole& R;
    LinShared<E, D>& sh;
    uint32_t base;
    int stream, seg, b, h, n, first, last, stop, delta;
    bool rev;
    float lg;

    __device__ __forceinline__ uint32_t tile(int stage, int k) const   // k: 0 a, 1 b, 2 c
    {
        return base + (STATE_ONLY ? stage * 2 + k - 1 : stage * 3 + k) * L::kTile;
    }
    __device__ __forceinline__ uint32_t state() const { return base + L::kStages * 3 * L::kTile; }
    __device__ __forceinline__ float gpow(int k) const { return exp2f(lg * static_cast<float>(k)); }
    __device__ __forceinline__ GroupLoader<E, D> loader(const void* t, long long ld, int warp) const
    {
        return GroupLoader<E, D>(t, ld, static_cast<long long>(b) * p.T, h * D, first + 16 * warp, n, rev);
    }
};

// ------------------------------------------------------------- state warps
template <typename E, int D, bool STATE_ONLY>
__device__ __forceinline__ void state_warp(const LinWork<E, D, STATE_ONLY>& W, int warp)
{
    using L = LinTile<E, D>;
    constexpr int NI = L::NI, NM = L::NM, NT = D / 8, UNROLL = 128 / D;
    const LinParams& p = W.p;
    const LinRole& R = W.R;
    const int lane = threadIdx.x & 31, r4 = lane >> 2, x2 = 2 * (lane & 3);
    const int lm_row = (lane & 7) + ((lane >> 4) << 3), lm_c = (lane >> 3) & 1;   // blocks (0,0) (0,1) (1,0) (1,1)
    const int lt_row = (lane & 7) + (((lane >> 3) & 1) << 3), lt_c = lane >> 4;   // blocks (0,0) (1,0) (0,1) (1,1)
    GroupLoader<E, D> lb = W.loader(R.b, R.ldb, warp);
#pragma unroll
    for (int s = 0; s < L::kStages - 1; ++s) {
        if (W.first + s * D < W.stop) lb.next(W.tile(s, 1) + warp * L::kGroup, W.n);
        cp_async_commit();
    }

    // the state at the segment's start, rows 16 warp + r4 (+ 8), columns 8 t + x2 (+ 1)
    float X[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) X[t][0] = X[t][1] = X[t][2] = X[t][3] = 0.f;
    const size_t mat = static_cast<size_t>(W.stream) * D * D;
    auto add_state = [&](const float* m, bool transposed, float f) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
                const int i = 16 * warp + r4 + 4 * k, j = 8 * t + x2;
                const float2 v = transposed ? make_float2(m[j * D + i], m[(j + 1) * D + i])
                                            : *reinterpret_cast<const float2*>(m + i * D + j);
                X[t][k] = fmaf(f, v.x, X[t][k]);
                X[t][k + 1] = fmaf(f, v.y, X[t][k + 1]);
            }
    };
    float bound = 0.f;   // >= every |X|, the same in every state warp
    if constexpr (!STATE_ONLY) {
        if (p.segments > 1) griddep_wait();   // the earlier segments' states come from the kernel before
        const int before = min(W.first, W.n);
        if (R.x_in) add_state(R.x_in + mat, R.transposed, before > 0 ? W.gpow(before) : 1.f);   // as it is, whatever g
        // what the earlier segments with tokens left, in their order; several of their loads in flight at once
        const int filled = min(W.seg, (W.n + p.seg_len - 1) / p.seg_len);
        const float* left = p.seg_state + (static_cast<size_t>(R.state_slot) * p.segments * p.B * p.H + W.stream) * D * D;
#pragma unroll UNROLL
        for (int s = 0; s < filled; ++s)
            add_state(left + static_cast<size_t>(s) * p.B * p.H * D * D, R.state_transposed,
                      W.gpow(before - min((s + 1) * p.seg_len, W.n)));
        float m = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, fabsf(X[t][k]));
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        if (lane == 0) W.sh.top[warp] = m;
        named_sync(2, L::kThreads / 2);
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w) bound = fmaxf(bound, W.sh.top[w]);
    }
    // the copy for the output warps: X * 2^-e, at most 2^14
    auto store_state = [&]() {
        const int eb = max(static_cast<int>(__float_as_uint(bound) >> 23), 14);
        const float sc = bound == 0.f ? 0.f : pow2i(140 - eb);
        if (threadIdx.x == L::kThreads / 2) W.sh.state_exp = bound == 0.f ? kNoValue : eb - 140;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const uint32_t at = state_at<D>(W.state(), 16 * warp + r4 + 8 * k, t, 0) + 2 * x2;
                uint32_t hi, lo;
                if constexpr (NM == 2) {
                    split_half2(X[t][2 * k] * sc, X[t][2 * k + 1] * sc, hi, lo);
                    asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + L::kState), "r"(lo) : "memory");
                } else {
                    hi = pack_half2(X[t][2 * k] * sc, X[t][2 * k + 1] * sc);
                }
                asm volatile("st.shared.u32 [%0], %1;" ::"r"(at), "r"(hi) : "memory");
            }
    };
    if constexpr (!STATE_ONLY) store_state();

    float cf[4];   // g^(15 - x) for this lane's tokens x of a group
#pragma unroll
    for (int k = 0; k < 4; ++k) cf[k] = W.gpow(15 - (x2 + (k & 1) + 8 * (k >> 1)));
    const Decay full = decay_over(W.lg, D);
    const float g_group = W.gpow(16), g_delta = W.delta ? W.gpow(1) : 1.f;

    int stage = 0, ahead = L::kStages - 1;   // ahead: the stage that chunk c + kStages - 1 goes to
    for (int pos = W.first; pos < W.stop; pos += D) {
        const int nc = min(D, W.stop - pos);   // valid positions in the chunk
        cp_async_wait<L::kStages - 2>();
        const int eb_own = convert_group<E, D>(W.tile(stage, 1) + warp * L::kGroup);
        if (lane == 0) W.sh.exp[stage][0][warp] = eb_own;
        named_sync(3, L::kThreads);   // terms, exponents and the state's copy are in place; the stage before is free
        if (pos + (L::kStages - 1) * D < W.stop) lb.next(W.tile(ahead, 1) + warp * L::kGroup, W.n);
        cp_async_commit();

        // X = g^nc X + alpha_u sum_j g^(nc-1-j+delta) b_j c_j^T, the sum normalised to the largest group's exponent
        int e[L::kWarps];
        float top = -8000.f;
#pragma unroll
        for (int g = 0; g < L::kWarps; ++g) {
            e[g] = W.sh.exp[stage][0][g] + W.sh.exp[stage][1][g];
            top = fmaxf(top, fmaf(W.lg, static_cast<float>(max(0, nc - 16 * g - 16) + W.delta), static_cast<float>(e[g])));
        }
        int eu = static_cast<int>(ceilf(top));
        float U[NT][4];
#pragma unroll
        for (int t = 0; t < NT; ++t) U[t][0] = U[t][1] = U[t][2] = U[t][3] = 0.f;
        float to_end = g_delta;   // g^(tokens after the group, + delta)
#pragma unroll
        for (int g = L::kWarps - 1; g >= 0; --g) {
            const float f = pow2i(e[g] - eu);
            float wt[4];
            if (nc == D) {
#pragma unroll
                for (int k = 0; k < 4; ++k) wt[k] = f * to_end * cf[k];
                to_end *= g_group;
            } else {   // rows past nc are zeros, whatever their weight
#pragma unroll
                for (int k = 0; k < 4; ++k)
                    wt[k] = f * W.gpow(max(0, nc - 1 - (16 * g + x2 + (k & 1) + 8 * (k >> 1))) + W.delta);
            }
            uint32_t bt[NI][4], bh[4], bl[4];
#pragma unroll
            for (int k = 0; k < NI; ++k)
                ldmatrix4_trans(bt[k], tile_at<E, D>(W.tile(stage, 1), 16 * g + lm_row, 2 * warp + lm_c, k));
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                float2 v = unpack_half2(bt[0][k]);
                if constexpr (NI == 2) {
                    const float2 lo = unpack_half2(bt[1][k]);
                    v.x += lo.x;
                    v.y += lo.y;
                }
                split_half2_2(mul2(v, make_float2(wt[2 * (k >> 1)], wt[2 * (k >> 1) + 1])), bh[k], bl[k]);
            }
#pragma unroll
            for (int t = 0; t < NT; t += 2) {
                uint32_t vf[4];
                ldmatrix4_trans(vf, tile_at<E, D>(W.tile(stage, 2), 16 * g + lt_row, t + lt_c, 0));
                mma16816(U[t], bh, vf[0], vf[1]);
                mma16816(U[t + 1], bh, vf[2], vf[3]);
                mma16816(U[t], bl, vf[0], vf[1]);
                mma16816(U[t + 1], bl, vf[2], vf[3]);
                if constexpr (NI == 2) {
                    ldmatrix4_trans(vf, tile_at<E, D>(W.tile(stage, 2), 16 * g + lt_row, t + lt_c, 1));
                    mma16816(U[t], bh, vf[0], vf[1]);
                    mma16816(U[t + 1], bh, vf[2], vf[3]);
                }
            }
        }
        eu += R.alpha_u_exp;
        const int bound_exp = eu + 28;   // |U| < D 2^28
        if (eu < -60 || eu > 60) {       // in two steps where one factor would leave fp32's range
            const float f = pow2i(eu / 2);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) U[t][k] *= f;
            eu -= eu / 2;
        }
        const float fu = R.alpha_u_man * pow2i(eu);
        const Decay dec = nc == D ? full : decay_over(W.lg, nc);
        if (dec.c == 1.f) {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) X[t][k] = fmaf(U[t][k], fu, fmaf(X[t][k], dec.m, X[t][k]));
        } else {
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) X[t][k] = fmaf(U[t][k], fu, X[t][k] * dec.m);
        }
        if constexpr (!STATE_ONLY) {
            if (pos + D < W.stop) {
                const float most = fabsf(R.alpha_u_man) * pow2i(bound_exp / 2) * static_cast<float>(D) *
                                   pow2i(bound_exp - bound_exp / 2);
                bound = fminf(fmaf(bound, dec.m + dec.c, most) * 1.0001f, 1.7e38f);
                named_sync(1, L::kThreads);   // the output warps have read the copy
                store_state();
            }
        }
        stage = stage + 1 == L::kStages ? 0 : stage + 1;
        ahead = ahead + 1 == L::kStages ? 0 : ahead + 1;
    }

    if constexpr (STATE_ONLY) {
        float* m = p.seg_state + ((static_cast<size_t>(R.state_slot) * p.segments + W.seg) * p.B * p.H + W.stream) * D * D;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float2*>(m + (16 * warp + r4 + 8 * k) * D + 8 * t + x2) =
                    make_float2(X[t][2 * k], X[t][2 * k + 1]);
    } else if (R.x_out && W.last == p.T) {
        float* m = R.x_out + mat;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int i = 16 * warp + r4 + 8 * (k >> 1), j = 8 * t + x2 + (k & 1);
                m[R.transposed ? j * D + i : i * D + j] = X[t][k];
            }
    }
}

// ------------------------------------------------------------- output warps
template <typename E, int D, bool STATE_ONLY>
__device__ __forceinline__ void output_warp(const LinWork<E, D, STATE_ONLY>& W, int warp)
{
    using L = LinTile<E, D>;
    constexpr int NI = L::NI, NM = L::NM, KS = D / 16, NT = D / 8;
    const LinParams& p = W.p;
    const LinRole& R = W.R;
    const int lane = threadIdx.x & 31, r4 = lane >> 2, x2 = 2 * (lane & 3);
    const int lm_row = (lane & 7) + ((lane >> 4) << 3), lm_c = (lane >> 3) & 1;
    const int lt_row = (lane & 7) + (((lane >> 3) & 1) << 3), lt_c = lane >> 4;
    const int own = warp * L::kGroup;
    GroupLoader<E, D> la = W.loader(STATE_ONLY ? R.c : R.a, STATE_ONLY ? R.ldc : R.lda, warp);
    GroupLoader<E, D> lc = W.loader(R.c, R.ldc, warp);
    auto load = [&](int stage) {
        if constexpr (!STATE_ONLY) la.next(W.tile(stage, 0) + own, W.n);
        lc.next(W.tile(stage, 2) + own, W.n);
    };
#pragma unroll
    for (int s = 0; s < L::kStages - 1; ++s) {
        if (W.first + s * D < W.stop) load(s);
        cp_async_commit();
    }
    E* po = nullptr;
    float cf[4], dg[2][4], rho[2];   // g^(15 - x), g^(r - x) inside the diagonal block, g^r
    if constexpr (!STATE_ONLY) {
        po = static_cast<E*>(R.out) + static_cast<long long>(W.b) * p.T * R.ldo + W.h * D;
#pragma unroll
        for (int k = 0; k < 4; ++k) cf[k] = W.gpow(15 - (x2 + (k & 1) + 8 * (k >> 1)));
#pragma unroll
        for (int k = 0; k < 2; ++k) rho[k] = W.gpow(r4 + 8 * k);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int gap = r4 + 8 * (k >> 1) - (8 * t + x2 + (k & 1));
                dg[t][k] = gap >= 0 ? W.gpow(gap) : 0.f;
            }
    }
    const float to_state = W.lg * static_cast<float>(16 * warp + 1 - W.delta);
    const float g_state = exp2f(to_state), g_group = W.gpow(16), g_near = W.gpow(1);

    int stage = 0, ahead = L::kStages - 1;
    for (int pos = W.first; pos < W.stop; pos += D) {
        cp_async_wait<L::kStages - 2>();
        int ea = 0;
        if constexpr (!STATE_ONLY) ea = convert_group<E, D>(W.tile(stage, 0) + own);
        const int ec_own = convert_group<E, D>(W.tile(stage, 2) + own);
        if (lane == 0) W.sh.exp[stage][1][warp] = ec_own;
        named_sync(3, L::kThreads);   // terms, exponents and the state's copy are in place; the stage before is free
        if (pos + (L::kStages - 1) * D < W.stop) load(ahead);
        cp_async_commit();

        if constexpr (!STATE_ONLY) {
            const int eX = W.sh.state_exp;
            uint32_t qf[NI][KS][4];
#pragma unroll
            for (int k = 0; k < NI; ++k)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    ldmatrix4(qf[k][ks], tile_at<E, D>(W.tile(stage, 0), 16 * warp + lt_row, 2 * ks + lt_c, k));
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
            // a X
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t s[4];
                    ldmatrix4_trans(s, state_at<D>(W.state(), 16 * ks + lt_row, t + lt_c, 0));
                    mma16816(acc[t], qf[0][ks], s[0], s[1]);
                    mma16816(acc[t + 1], qf[0][ks], s[2], s[3]);
                    if constexpr (NI == 2) {
                        mma16816(acc[t], qf[1][ks], s[0], s[1]);
                        mma16816(acc[t + 1], qf[1][ks], s[2], s[3]);
                    }
                    if constexpr (NM == 2) {
                        ldmatrix4_trans(s, state_at<D>(W.state(), 16 * ks + lt_row, t + lt_c, 1));
                        mma16816(acc[t], qf[0][ks], s[0], s[1]);
                        mma16816(acc[t + 1], qf[0][ks], s[2], s[3]);
                    }
                }
            if (pos + D < W.stop) named_arrive(1, L::kThreads);   // the state's copy may change
            // One exponent ef for the strip: score columns of group g carry
            // alpha_u 2^(eb + ec) g^(gap) after 2^-20 (|a b| < 2^34 becomes < 2^15), the
            // state's part 2^(eX - 20); the largest of them becomes 1.
            float top = fmaxf(static_cast<float>(eX - 20) + to_state, -8000.f);
            auto exponent = [&](int g) { return W.sh.exp[stage][0][g] + W.sh.exp[stage][1][g] + R.alpha_u_exp; };
#pragma unroll
            for (int g = 0; g < L::kWarps; ++g)
                if (g <= warp)
                    top = fmaxf(top, fmaf(W.lg, static_cast<float>(g < warp ? 16 * (warp - g) - 15 : 0),
                                          static_cast<float>(exponent(g))));
            const int ef = static_cast<int>(ceilf(top));
            {
                const float f = g_state * pow2i(eX - 20 - ef);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[t][k] *= f * rho[k >> 1];
            }
            auto score = [&](float (&s)[2][4], int g) {   // a b^T of strip `warp` and group g
#pragma unroll
                for (int t = 0; t < 2; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kf[4];
                    ldmatrix4(kf, tile_at<E, D>(W.tile(stage, 1), 16 * g + lm_row, 2 * ks + lm_c, 0));
                    mma16816(s[0], qf[0][ks], kf[0], kf[1]);
                    mma16816(s[1], qf[0][ks], kf[2], kf[3]);
                    if constexpr (NI == 2) {
                        mma16816(s[0], qf[1][ks], kf[0], kf[1]);
                        mma16816(s[1], qf[1][ks], kf[2], kf[3]);
                        ldmatrix4(kf, tile_at<E, D>(W.tile(stage, 1), 16 * g + lm_row, 2 * ks + lm_c, 1));
                        mma16816(s[0], qf[0][ks], kf[0], kf[1]);
                        mma16816(s[1], qf[0][ks], kf[2], kf[3]);
                    }
                }
            };
            auto apply = [&](const float (&s)[2][4], int g) {   // acc += s c of group g
                uint32_t ph[4], pl[4];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        if constexpr (NM == 2)
                            split_half2(s[t][2 * k], s[t][2 * k + 1], ph[2 * t + k], pl[2 * t + k]);
                        else
                            ph[2 * t + k] = pack_half2(s[t][2 * k], s[t][2 * k + 1]);
                    }
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t vf[4];
                    ldmatrix4_trans(vf, tile_at<E, D>(W.tile(stage, 2), 16 * g + lt_row, t + lt_c, 0));
                    mma16816(acc[t], ph, vf[0], vf[1]);
                    mma16816(acc[t + 1], ph, vf[2], vf[3]);
                    if constexpr (NM == 2) {
                        mma16816(acc[t], pl, vf[0], vf[1]);
                        mma16816(acc[t + 1], pl, vf[2], vf[3]);
                    }
                    if constexpr (NI == 2) {
                        ldmatrix4_trans(vf, tile_at<E, D>(W.tile(stage, 2), 16 * g + lt_row, t + lt_c, 1));
                        mma16816(acc[t], ph, vf[0], vf[1]);
                        mma16816(acc[t + 1], ph, vf[2], vf[3]);
                    }
                }
            };
            {
                float s[2][4];
                score(s, warp);
                const float f = pow2i(exponent(warp) - 20 - ef) * R.alpha_u_man;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[t][k] *= f * dg[t][k];
                apply(s, warp);
            }
            float near = g_near;   // g^(16 (warp - g) - 15)
#pragma unroll 1
            for (int g = warp - 1; g >= 0; --g) {
                float s[2][4];
                score(s, g);
                const float f = near * R.alpha_u_man * pow2i(exponent(g) - 20 - ef);
                near *= g_group;
                const float f0 = f * rho[0], f1 = f * rho[1];
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[t][k] *= (k < 2 ? f0 : f1) * cf[2 * t + (k & 1)];
                apply(s, g);
            }
            // out = alpha_o acc 2^(ea + ef + 20), in two steps where one factor would leave fp32's range
            int eo = ea + ef + 20;
            if (eo < -100 || eo > 100) {
                const float f = pow2i(eo / 2);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[t][k] *= f;
                eo -= eo / 2;
            }
            const float f = pow2i(eo) * R.alpha_o;
            const int i0 = pos + 16 * warp;
            if constexpr (sizeof(E) == 4) {
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = i0 + r4 + 8 * k;
                    if (i < W.stop) {
                        float* o = po + static_cast<long long>(W.rev ? W.n - 1 - i : i) * R.ldo + x2;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            *reinterpret_cast<float2*>(o + 8 * t) = make_float2(acc[t][2 * k] * f, acc[t][2 * k + 1] * f);
                    }
                }
            } else {
                // through the warp's own rows of a's tile (its fragments are in registers), then 16 bytes a lane
                __syncwarp();
                const uint32_t at = W.tile(stage, 0) + own;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = r4 + 8 * k;
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(at + r * L::kRow + (swizzle<D>(r, t) << 4) + 2 * x2),
                                     "r"(pack_pair(acc[t][2 * k] * f, acc[t][2 * k + 1] * f, E{}))
                                     : "memory");
                    }
                __syncwarp();
#pragma unroll
                for (int q = 0; q < L::kPieces; ++q) {
                    const int piece = lane + 32 * q, r = piece / L::kPerRow, c = piece % L::kPerRow, i = i0 + r;
                    uint4 v;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(at + r * L::kRow + (swizzle<D>(r, c) << 4)));
                    if (i < W.stop)
                        *reinterpret_cast<uint4*>(po + static_cast<long long>(W.rev ? W.n - 1 - i : i) * R.ldo + 8 * c) = v;
                }
            }
        }
        stage = stage + 1 == L::kStages ? 0 : stage + 1;
        ahead = ahead + 1 == L::kStages ? 0 : ahead + 1;
    }
    if constexpr (!STATE_ONLY) {
        // rows past the sequence's length
        const int z0 = max(W.first, W.n);
        const long long pieces = static_cast<long long>(W.last - z0) * L::kPerRow;
        for (long long q = threadIdx.x; q < pieces; q += L::kThreads / 2)
            *reinterpret_cast<uint4*>(po + (z0 + q / L::kPerRow) * R.ldo +
                                      q % L::kPerRow * (16 / static_cast<int>(sizeof(E)))) = make_uint4(0, 0, 0, 0);
    }
}

// STATE_ONLY: only X's update, from X = 0, for the segments before the last;
// X goes to seg_state (see LinParams).
template <typename E, int D, bool STATE_ONLY>
__device__ __forceinline__ void linattn_body(const LinParams& p)
{
    using L = LinTile<E, D>;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ LinShared<E, D> shared;
    const int streams = p.B * p.H;
    LinWork<E, D, STATE_ONLY> W{p, p.role[STATE_ONLY ? p.state_role[blockIdx.y] : blockIdx.y], shared, smem_u32(smem)};
    W.stream = blockIdx.x % streams;
    W.seg = blockIdx.x / streams;
    W.b = W.stream / p.H;
    W.h = W.stream % p.H;
    W.n = p.lengths ? min(max(p.lengths[W.b], 0), p.T) : p.T;
    W.first = W.seg * p.seg_len;
    W.last = p.T - W.first < p.seg_len ? p.T : W.first + p.seg_len;
    W.stop = min(W.last, W.n);   // positions at and past it are not processed
    W.rev = W.R.reverse != 0;
    W.delta = W.rev ? 1 : 0;
    W.lg = decay_log2(p.log_decay[W.h]);
    const int warp = threadIdx.x >> 5;
    if (warp < L::kWarps)
        output_warp(W, warp);
    else
        state_warp(W, warp - L::kWarps);
}

}  // namespace srwm
