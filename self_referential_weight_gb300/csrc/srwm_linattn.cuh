// srwm_linattn.cuh -- the chunked kernel of the primitive in srwm_linattn.h.
//
// One CTA runs one stream (sequence, head) of one role, or one segment of its
// length, in chunks of D tokens, with the D x D state X in registers: D / 16
// warps, warp w holding rows 16w .. 16w + 15 of X as accumulator fragments in
// fp32.  Per chunk (i, j positions in it, P = a b^T, g the decay):
//   out_i = alpha [ g^(i+1-delta) a_i X  +  sum_{j<=i} g^(i-j) P_ij c_j ]
//   X     = g^n X + alpha_u sum_j g^(n-1-j+delta) b_j c_j^T
// (delta = 0 in order, 1 in reverse).  Warp w computes output rows 16w .. + 15:
// a X from the state's fp16 copy in shared memory, then the columns j < 16w
// with the row's part of the decay taken out (g^(i-j) = g^(i-16w) g^(16w-j)),
// one multiplication by g^(i-16w), and the diagonal 16 x 16 block.  Blocks
// above the diagonal are not computed.
//
// The products run on the tensor cores in fp16 (mma.sync), with fp32 sums.
// Chunk of D tokens: the work per token is about 4 D^2 + 2.5 D^2 multiply-adds
// whatever T is, and a warp's share of every matrix is a 16-row strip.
//
// Range and precision.  Each group of 16 tokens of a, b and c is scaled by a
// power of two that puts its largest magnitude into [2^13, 2^14), exactly; all
// later factors carry exponents as integers and are normalised to the largest
// one in use, so fp16's range never matters.  fp32 values are split into a high
// and a low fp16 (22 bits); three of the four products are kept.  bf16 and
// fp16 values are one fp16 exactly.  The weighted rows of b always enter the
// state as pairs, so the state is good to fp32 for every type.  The score P
// and the state's copy enter their products as pairs for fp32 and fp16, and as
// one fp16 (2^-11 of each value) for bf16, whose outputs round by 2^-8.
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

// log2 of the decay per token: <= 0 and finite, so that multiples of it are.
__device__ __forceinline__ float decay_log2(float log_decay)
{
    return fmaxf(fminf(log_decay, 0.f) * 1.4426950408889634f, -16384.f);
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
    static constexpr int kWarps = D / 16;
    static constexpr int kThreads = 32 * kWarps;
    static constexpr int NI = sizeof(E) == 4 ? 2 : 1;                       // fp16 terms of an input
    static constexpr int NM = std::is_same<E, __nv_bfloat16>::value ? 1 : 2;  // of a score or the state's copy
    static constexpr int kRow = 2 * D;                                      // bytes of a row of one term
    static constexpr int kGroup = 16 * D * static_cast<int>(sizeof(E));      // 16 tokens: raw, later their terms
    static constexpr int kTile = kWarps * kGroup;                           // D tokens
    static constexpr int kState = D * kRow;                                 // one term of the state's copy
    static constexpr int kSmem = 2 * 3 * kTile + NM * kState;
    static constexpr int kSmemState = 2 * 2 * kTile;                        // the state-only pass
    static constexpr int kPieces = kGroup / 512;                            // 16-byte pieces per lane and group
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

// Starts the copy of this warp's 16 rows of one tensor.  pos: position of the
// group's first row; rows at or past n read nothing and become zeros.
template <typename E, int D>
__device__ __forceinline__ void load_group(uint32_t group, const E* stream, long long ld, int pos, int n, bool reverse)
{
    using L = LinTile<E, D>;
    const int lane = threadIdx.x & 31;
    constexpr int per_row = D * static_cast<int>(sizeof(E)) / 16;
#pragma unroll
    for (int q = 0; q < L::kPieces; ++q) {
        const int p = lane + 32 * q, r = p / per_row, c = p % per_row;
        const int i = pos + r;
        const bool ok = i < n;
        const long long t = ok ? (reverse ? n - 1 - i : i) : 0;
        const E* src = stream + t * ld + c * (16 / static_cast<int>(sizeof(E)));
        // 16-bit types land where their fp16 values will stay; fp32 rows lie plain until they are split
        const uint32_t dst = sizeof(E) == 2 ? group + r * L::kRow + (swizzle<D>(r, c) << 4) : group + p * 16;
        cp_async16(dst, src, ok);
    }
}

__device__ __forceinline__ float2 pair_to_f(uint32_t v, __nv_bfloat16)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
__device__ __forceinline__ float2 pair_to_f(uint32_t v, __half) { return unpack_half2(v); }

// Turns this warp's landed group into scaled fp16 terms in place.  Every lane
// converts the pieces it copied.  Returns the exponent e of the group: value = term * 2^e.
template <typename E, int D>
__device__ __forceinline__ int convert_group(uint32_t group)
{
    using L = LinTile<E, D>;
    const int lane = threadIdx.x & 31;
    constexpr int per_row = D * static_cast<int>(sizeof(E)) / 16;
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
                const float2 f = pair_to_f(v[q][k], E{});
                v[q][k] = pack_half2(f.x * sc, f.y * sc);
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

// STATE_ONLY: only X's update, from X = 0, for the segments before the last;
// X goes to seg_state (see linattn_plan).
template <typename E, int D, bool STATE_ONLY>
__device__ __forceinline__ void linattn_body(const LinParams& p)
{
    using L = LinTile<E, D>;
    constexpr int NI = L::NI, NM = L::NM, KS = D / 16, NT = D / 8;
    extern __shared__ __align__(128) unsigned char smem[];
    __shared__ int s_exp[2][3][L::kWarps];
    __shared__ float s_max[L::kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r4 = lane >> 2, x2 = 2 * (lane & 3);
    const int stream = blockIdx.x % (p.B * p.H), seg = blockIdx.x / (p.B * p.H);
    const int b = stream / p.H, h = stream % p.H;
    const LinRole& R = p.role[STATE_ONLY ? p.state_role[blockIdx.y] : blockIdx.y];
    const int n = p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    const int first = seg * p.seg_len, last = p.T - first < p.seg_len ? p.T : first + p.seg_len;   // its positions
    const bool rev = R.reverse != 0;
    const int delta = rev ? 1 : 0;
    const float lg = decay_log2(p.log_decay[h]);
    constexpr int kTensors = STATE_ONLY ? 2 : 3;
    const uint32_t base = smem_u32(smem);
    const uint32_t s_state = base + 2 * 3 * L::kTile;
    auto tile = [&](int buf, int k) { return base + (buf * kTensors + (STATE_ONLY ? k - 1 : k)) * L::kTile; };
    const long long tok0 = static_cast<long long>(b) * p.T;
    const E* pa = static_cast<const E*>(R.a) + tok0 * R.lda + h * D;
    const E* pb = static_cast<const E*>(R.b) + tok0 * R.ldb + h * D;
    const E* pc = static_cast<const E*>(R.c) + tok0 * R.ldc + h * D;
    const int stop = min(last, n);   // positions at and past it are not processed
    auto load = [&](int buf, int pos) {
        const int w0 = warp * L::kGroup, at = pos + 16 * warp;
        if constexpr (!STATE_ONLY) load_group<E, D>(tile(buf, 0) + w0, pa, R.lda, at, n, rev);
        load_group<E, D>(tile(buf, 1) + w0, pb, R.ldb, at, n, rev);
        load_group<E, D>(tile(buf, 2) + w0, pc, R.ldc, at, n, rev);
        cp_async_commit();
    };
    if (first < stop) load(0, first);

    // the state at the segment's start, rows 16 warp + r4 (+ 8), columns 8 t + x2 (+ 1)
    float X[NT][4];
#pragma unroll
    for (int t = 0; t < NT; ++t) X[t][0] = X[t][1] = X[t][2] = X[t][3] = 0.f;
    const size_t mat = static_cast<size_t>(stream) * D * D;
    auto element = [&](const float* m, int i, int j, bool transposed) { return transposed ? m[j * D + i] : m[i * D + j]; };
    auto add_state = [&](const float* m, bool transposed, float f) {
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k)
                X[t][k] = fmaf(f, element(m, 16 * warp + r4 + 8 * (k >> 1), 8 * t + x2 + (k & 1), transposed), X[t][k]);
    };
    float bound = 0.f;   // >= every |X|, the same in every warp
    if constexpr (!STATE_ONLY) {
        if (R.x_in) add_state(R.x_in + mat, R.transposed, exp2f(lg * static_cast<float>(min(first, n))));
        for (int s = 0; s < seg; ++s)   // what the earlier segments left, in their order
            add_state(p.seg_state + ((static_cast<size_t>(R.state_slot) * p.segments + s) * p.B * p.H + stream) * D * D,
                      R.state_transposed, exp2f(lg * static_cast<float>(min(first, n) - min((s + 1) * p.seg_len, n))));
        float m = 0.f;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) m = fmaxf(m, fabsf(X[t][k]));
        m = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(m)));
        if (lane == 0) s_max[warp] = m;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < L::kWarps; ++w) bound = fmaxf(bound, s_max[w]);
    }

    // decay factors that stay the same: g^(15 - x) for this lane's columns x of a
    // 16-column group, g^(r - x) inside the diagonal block, g^r
    float cf[4], dg[2][4], rho[2];
    auto gpow = [&](int k) { return exp2f(lg * static_cast<float>(k)); };
#pragma unroll
    for (int k = 0; k < 4; ++k) cf[k] = gpow(15 - (x2 + (k & 1) + 8 * (k >> 1)));
    if constexpr (!STATE_ONLY) {
        rho[0] = gpow(r4);
        rho[1] = gpow(r4 + 8);
#pragma unroll
        for (int t = 0; t < 2; ++t)
#pragma unroll
            for (int k = 0; k < 4; ++k) {
                const int gap = r4 + 8 * (k >> 1) - (8 * t + x2 + (k & 1));
                dg[t][k] = gap >= 0 ? gpow(gap) : 0.f;
            }
    }
    const Decay full = decay_over(lg, D);

    // the state's copy for the tensor cores: X * 2^-eX, at most 2^14
    int eX = kNoValue;
    auto store_state = [&]() {
        const int eb = max(static_cast<int>(__float_as_uint(bound) >> 23), 14);
        eX = bound == 0.f ? kNoValue : eb - 140;
        const float sc = bound == 0.f ? 0.f : pow2i(-eX);
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int r = 16 * warp + r4 + 8 * k;
                const uint32_t at = state_at<D>(s_state, r, t, 0) + 2 * x2;
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

    E* po = nullptr;
    if constexpr (!STATE_ONLY) po = static_cast<E*>(R.out) + tok0 * R.ldo + h * D;
    // lane addresses of the fragment loads: row and piece of each 8x8 block
    const int lm_row = (lane & 7) + ((lane >> 4) << 3), lm_c = (lane >> 3) & 1;        // blocks (0,0) (0,1) (1,0) (1,1)
    const int lt_row = (lane & 7) + (((lane >> 3) & 1) << 3), lt_c = lane >> 4;        // blocks (0,0) (1,0) (0,1) (1,1)

    int buf = 0;
    for (int pos = first; pos < stop; pos += D, buf ^= 1) {
        const int nc = min(D, stop - pos);   // valid positions in the chunk
        cp_async_wait<0>();
        const int w0 = warp * L::kGroup;
        int ea = 0;
        if constexpr (!STATE_ONLY) ea = convert_group<E, D>(tile(buf, 0) + w0);
        const int eb_own = convert_group<E, D>(tile(buf, 1) + w0);
        const int ec_own = convert_group<E, D>(tile(buf, 2) + w0);
        if (lane == 0) {
            s_exp[buf][1][warp] = eb_own;
            s_exp[buf][2][warp] = ec_own;
        }
        __syncthreads();   // terms, exponents and the state's copy are in place; the other buffer is free
        if (pos + D < stop) load(buf ^ 1, pos + D);

        if constexpr (!STATE_ONLY) {
            uint32_t qf[NI][KS][4];
#pragma unroll
            for (int k = 0; k < NI; ++k)
#pragma unroll
                for (int ks = 0; ks < KS; ++ks)
                    ldmatrix4(qf[k][ks], tile_at<E, D>(tile(buf, 0), 16 * warp + lt_row, 2 * ks + lt_c, k));
            float acc[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;
            // a X
#pragma unroll
            for (int ks = 0; ks < KS; ++ks)
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t s[4];
                    ldmatrix4_trans(s, state_at<D>(s_state, 16 * ks + lt_row, t + lt_c, 0));
                    mma16816(acc[t], qf[0][ks], s[0], s[1]);
                    mma16816(acc[t + 1], qf[0][ks], s[2], s[3]);
                    if constexpr (NI == 2) {
                        mma16816(acc[t], qf[1][ks], s[0], s[1]);
                        mma16816(acc[t + 1], qf[1][ks], s[2], s[3]);
                    }
                    if constexpr (NM == 2) {
                        ldmatrix4_trans(s, state_at<D>(s_state, 16 * ks + lt_row, t + lt_c, 1));
                        mma16816(acc[t], qf[0][ks], s[0], s[1]);
                        mma16816(acc[t + 1], qf[0][ks], s[2], s[3]);
                    }
                }
            // One exponent ef for the strip: score columns of group g carry
            // alpha_u 2^(eb + ec) g^(gap) after 2^-20 (|a b| < 2^34 becomes < 2^15), the
            // state's part 2^(eX - 20); the largest of them becomes 1.
            const float to_state = lg * static_cast<float>(16 * warp + 1 - delta);
            float top = static_cast<float>(eX - 20) + to_state;
#pragma unroll
            for (int g = 0; g < L::kWarps; ++g)
                if (g <= warp)
                    top = fmaxf(top, static_cast<float>(s_exp[buf][1][g] + s_exp[buf][2][g] + R.alpha_u_exp) +
                                         lg * static_cast<float>(g < warp ? 16 * (warp - g) - 15 : 0));
            const int ef = static_cast<int>(ceilf(fmaxf(top, -8000.f)));
            {
                const float f = exp2f(to_state) * pow2i(eX - 20 - ef);
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) acc[t][k] *= f;
            }
            auto score = [&](float (&s)[2][4], int g) {   // a b^T of strip `warp` and group g
#pragma unroll
                for (int t = 0; t < 2; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
#pragma unroll
                for (int ks = 0; ks < KS; ++ks) {
                    uint32_t kf[4];
                    ldmatrix4(kf, tile_at<E, D>(tile(buf, 1), 16 * g + lm_row, 2 * ks + lm_c, 0));
                    mma16816(s[0], qf[0][ks], kf[0], kf[1]);
                    mma16816(s[1], qf[0][ks], kf[2], kf[3]);
                    if constexpr (NI == 2) {
                        mma16816(s[0], qf[1][ks], kf[0], kf[1]);
                        mma16816(s[1], qf[1][ks], kf[2], kf[3]);
                        ldmatrix4(kf, tile_at<E, D>(tile(buf, 1), 16 * g + lm_row, 2 * ks + lm_c, 1));
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
                    ldmatrix4_trans(vf, tile_at<E, D>(tile(buf, 2), 16 * g + lt_row, t + lt_c, 0));
                    mma16816(acc[t], ph, vf[0], vf[1]);
                    mma16816(acc[t + 1], ph, vf[2], vf[3]);
                    if constexpr (NM == 2) {
                        mma16816(acc[t], pl, vf[0], vf[1]);
                        mma16816(acc[t + 1], pl, vf[2], vf[3]);
                    }
                    if constexpr (NI == 2) {
                        ldmatrix4_trans(vf, tile_at<E, D>(tile(buf, 2), 16 * g + lt_row, t + lt_c, 1));
                        mma16816(acc[t], ph, vf[0], vf[1]);
                        mma16816(acc[t + 1], ph, vf[2], vf[3]);
                    }
                }
            };
#pragma unroll 1
            for (int g = 0; g < warp; ++g) {
                float s[2][4];
                score(s, g);
                const float f = gpow(16 * (warp - g) - 15) * R.alpha_u_man *
                                pow2i(s_exp[buf][1][g] + s_exp[buf][2][g] + R.alpha_u_exp - 20 - ef);
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[t][k] *= f * cf[2 * t + (k & 1)];
                apply(s, g);
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) acc[t][k] *= rho[k >> 1];
            {
                float s[2][4];
                score(s, warp);
                const float f = pow2i(eb_own + ec_own + R.alpha_u_exp - 20 - ef) * R.alpha_u_man;
#pragma unroll
                for (int t = 0; t < 2; ++t)
#pragma unroll
                    for (int k = 0; k < 4; ++k) s[t][k] *= f * dg[t][k];
                apply(s, warp);
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
                    if (i < stop) {
                        float* o = po + static_cast<long long>(rev ? n - 1 - i : i) * R.ldo + x2;
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            *reinterpret_cast<float2*>(o + 8 * t) = make_float2(acc[t][2 * k] * f, acc[t][2 * k + 1] * f);
                    }
                }
            } else {
                // through the warp's own rows of a's tile (its fragments are in registers), then 16 bytes a lane
                __syncwarp();
                const uint32_t own = tile(buf, 0) + w0;
#pragma unroll
                for (int t = 0; t < NT; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int r = r4 + 8 * k;
                        E two[2] = {from_f<E>(acc[t][2 * k] * f), from_f<E>(acc[t][2 * k + 1] * f)};
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(own + r * L::kRow + (swizzle<D>(r, t) << 4) + 2 * x2),
                                     "r"(*reinterpret_cast<const uint32_t*>(two))
                                     : "memory");
                    }
                __syncwarp();
                constexpr int per_row = D / 8;
#pragma unroll
                for (int q = 0; q < L::kPieces; ++q) {
                    const int pc16 = lane + 32 * q, r = pc16 / per_row, c = pc16 % per_row, i = i0 + r;
                    uint4 v;
                    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                                 : "r"(own + r * L::kRow + (swizzle<D>(r, c) << 4)));
                    if (i < stop)
                        *reinterpret_cast<uint4*>(po + static_cast<long long>(rev ? n - 1 - i : i) * R.ldo + 8 * c) = v;
                }
            }
        }

        // X = g^nc X + alpha_u sum_j g^(nc-1-j+delta) b_j c_j^T
        {
            float top = -8000.f;
#pragma unroll
            for (int g = 0; g < L::kWarps; ++g)
                top = fmaxf(top, static_cast<float>(s_exp[buf][1][g] + s_exp[buf][2][g]) +
                                     lg * static_cast<float>(max(0, nc - 16 * g - 16) + delta));
            int eu = static_cast<int>(ceilf(top));
            float U[NT][4];
#pragma unroll
            for (int t = 0; t < NT; ++t) U[t][0] = U[t][1] = U[t][2] = U[t][3] = 0.f;
#pragma unroll
            for (int g = 0; g < L::kWarps; ++g) {
                const float f = pow2i(s_exp[buf][1][g] + s_exp[buf][2][g] - eu);
                float wt[4];
                if (nc == D) {
                    const float fg = f * gpow(D - 16 * g - 16 + delta);
#pragma unroll
                    for (int k = 0; k < 4; ++k) wt[k] = fg * cf[k];
                } else {   // rows past nc are zeros, whatever their weight
#pragma unroll
                    for (int k = 0; k < 4; ++k)
                        wt[k] = f * gpow(max(0, nc - 1 - (16 * g + x2 + (k & 1) + 8 * (k >> 1))) + delta);
                }
                uint32_t bt[NI][4], bh[4], bl[4];
#pragma unroll
                for (int k = 0; k < NI; ++k)
                    ldmatrix4_trans(bt[k], tile_at<E, D>(tile(buf, 1), 16 * g + lm_row, 2 * warp + lm_c, k));
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    float2 v = unpack_half2(bt[0][k]);
                    if constexpr (NI == 2) {
                        const float2 lo = unpack_half2(bt[1][k]);
                        v.x += lo.x;
                        v.y += lo.y;
                    }
                    split_half2(v.x * wt[2 * (k >> 1)], v.y * wt[2 * (k >> 1) + 1], bh[k], bl[k]);
                }
#pragma unroll
                for (int t = 0; t < NT; t += 2) {
                    uint32_t vf[4];
                    ldmatrix4_trans(vf, tile_at<E, D>(tile(buf, 2), 16 * g + lt_row, t + lt_c, 0));
                    mma16816(U[t], bh, vf[0], vf[1]);
                    mma16816(U[t + 1], bh, vf[2], vf[3]);
                    mma16816(U[t], bl, vf[0], vf[1]);
                    mma16816(U[t + 1], bl, vf[2], vf[3]);
                    if constexpr (NI == 2) {
                        ldmatrix4_trans(vf, tile_at<E, D>(tile(buf, 2), 16 * g + lt_row, t + lt_c, 1));
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
            const Decay dec = nc == D ? full : decay_over(lg, nc);
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) X[t][k] = fmaf(X[t][k], dec.m, fmaf(U[t][k], fu, X[t][k] * dec.c));
            if constexpr (!STATE_ONLY) {
                const float most = fabsf(R.alpha_u_man) * pow2i(bound_exp / 2) * static_cast<float>(D) *
                                   pow2i(bound_exp - bound_exp / 2);
                bound = fminf(fmaf(bound, dec.m + dec.c, most) * 1.0001f, 1.7e38f);
                if (pos + D < stop) {
                    __syncthreads();   // every warp is done with the state's copy
                    store_state();
                }
            }
        }
    }

    if constexpr (STATE_ONLY) {
        float* m = p.seg_state + ((static_cast<size_t>(R.state_slot) * p.segments + seg) * p.B * p.H + stream) * D * D;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int k = 0; k < 2; ++k)
                *reinterpret_cast<float2*>(m + (16 * warp + r4 + 8 * k) * D + 8 * t + x2) =
                    make_float2(X[t][2 * k], X[t][2 * k + 1]);
    } else {
        if (R.x_out && last == p.T) {
            float* m = R.x_out + mat;
#pragma unroll
            for (int t = 0; t < NT; ++t)
#pragma unroll
                for (int k = 0; k < 4; ++k) {
                    const int i = 16 * warp + r4 + 8 * (k >> 1), j = 8 * t + x2 + (k & 1);
                    m[R.transposed ? j * D + i : i * D + j] = X[t][k];
                }
        }
        // rows past the sequence's length
        constexpr int per_row = D * static_cast<int>(sizeof(E)) / 16;
        const int z0 = max(first, n), pieces = (last - z0) * per_row;
        for (int q = threadIdx.x; q < pieces; q += L::kThreads)
            *reinterpret_cast<uint4*>(po + static_cast<long long>(z0 + q / per_row) * R.ldo +
                                      (q % per_row) * (16 / static_cast<int>(sizeof(E)))) = make_uint4(0, 0, 0, 0);
    }
}

}  // namespace srwm
