// srwm_linattn_scan.cu -- the primitive of srwm_linattn.h token by token, for
// short sequences: the state stays in registers, in fp32 throughout.
//
//   H_i = f_i H_{i-1} + (alpha_u c_i) b_i,   out_i = alpha_o (a_i . H_i)
// per column of the state, f_i = g, or 1 for the first token in reverse.  A
// thread holds one column, so no sum crosses threads; a and b are read from
// shared memory by all of a stream's D threads at once.  That is 1.5 D two-wide
// fp32 operations a token, against a whole chunk of D (or 128) tokens in the
// chunked kernels however few of them there are.
//
// What bounds it: at D = 64 shared memory, from which every warp loads a token's a
// and b in full (2048 streams, gradients, T = 40: 130 us, with L1 at 86 % of its rate, the
// fp32 pipe at 62 % and three warps on a scheduler), and below T = 10 the states,
// read and written once (T = 1: 34 us for 134 MB); at D = 16 a token's latency, about 0.1 us.  Several
// tokens are unrolled so that one's loads run under another's sums (d = 16, 2048
// streams of 26 tokens in fp32: 7.5 us one by one, 6.4 by four).
#include <cuda_runtime.h>

#include "srwm_check.h"
#include "srwm_f2.cuh"
#include "srwm_linattn.cuh"
#include "srwm_linattn_scan.h"

namespace srwm {
namespace {

constexpr int kThreads = 128;
constexpr int TT = 8;        // tokens of a tile
constexpr int STAGES = 3;    // tiles in flight

template <typename E, int D>
struct ScanTile {
    static constexpr int kStreams = kThreads / D;                     // of a CTA
    static constexpr int kRow = D * static_cast<int>(sizeof(E));      // bytes of a token's row
    static constexpr int kPerRow = kRow / 16;
    static constexpr int kTile = 3 * TT * kRow;                       // a | b | c as they land
    static constexpr int kWide = sizeof(E) == 4 ? 0 : 3 * TT * D * 4; // and as fp32, two of them
    static constexpr int kStream = STAGES * kTile + 2 * kWide + (D == 16 ? 64 : 0);   // a warp's two streams: other banks
    static constexpr int kSmem = kStreams * kStream;
};

template <typename E, int D>
__global__ void __launch_bounds__(kThreads) linattn_scan_kernel(const __grid_constant__ LinParams p)
{
    using L = ScanTile<E, D>;
    constexpr int UNROLL = D == 64 ? 2 : 4;
    extern __shared__ __align__(128) unsigned char smem[];
    const LinRole& R = p.role[blockIdx.y];
    const int local = threadIdx.x / D, col = threadIdx.x % D;
    const int streams = p.B * p.H, stream = blockIdx.x * L::kStreams + local;
    const bool on = stream < streams;
    const int b = on ? stream / p.H : 0, h = on ? stream % p.H : 0;
    const int n = !on ? 0 : p.lengths ? min(max(p.lengths[b], 0), p.T) : p.T;
    // two streams of D = 16 share a warp and run as long as the longer one
    const int steps = D == 16 ? max(n, __shfl_xor_sync(0xffffffffu, n, 16)) : n;
    const bool rev = R.reverse != 0;
    auto meet = [&]() {   // the stream's threads
        if constexpr (D == 64)
            named_sync(1 + local, 64);
        else
            __syncwarp();
    };
    const uint32_t base = smem_u32(smem) + local * L::kStream;
    const E* const in[3] = {static_cast<const E*>(R.a), static_cast<const E*>(R.b), static_cast<const E*>(R.c)};
    const long long ld[3] = {R.lda, R.ldb, R.ldc};
    const long long token0 = static_cast<long long>(b) * p.T;
    auto load = [&](int tile) {   // positions TT * tile ..; those at or past n become zeros
        const uint32_t to = base + tile % STAGES * L::kTile;
#pragma unroll
        for (int k = 0; k < 3; ++k)
#pragma unroll
            for (int q = 0; q < TT * L::kPerRow; q += D) {
                const int piece = q + col, r = piece / L::kPerRow, i = TT * tile + r;
                const bool ok = i < n;
                const E* from = in[k] + (token0 + (ok ? (rev ? n - 1 - i : i) : 0)) * ld[k] + h * D;
                cp_async16(to + k * TT * L::kRow + piece * 16, from + (ok ? piece % L::kPerRow * (16 / sizeof(E)) : 0), ok);
            }
    };
    const int tiles = (steps + TT - 1) / TT;
#pragma unroll
    for (int s = 0; s < STAGES - 1; ++s) {
        if (s < tiles) load(s);
        cp_async_commit();
    }

    const size_t mat = static_cast<size_t>(on ? stream : 0) * D * D;
    float2 X[D / 2];   // column `col`, rows 2 i and 2 i + 1
#pragma unroll
    for (int i = 0; i < D / 2; ++i) X[i] = both(0.f);
    if (R.x_in && on) {
        const float* x = R.x_in + mat + (R.transposed ? col * D : col);
#pragma unroll
        for (int i = 0; i < D / 2; i += 2) {
            const float* y = x + 2 * i * D;
            const float4 v = R.transposed ? *reinterpret_cast<const float4*>(x + 2 * i)
                                          : make_float4(y[0], y[D], y[2 * D], y[3 * D]);
            X[i] = make_float2(v.x, v.y);
            X[i + 1] = make_float2(v.z, v.w);
        }
    }
    // A token's decay in fp32 takes up what the roundings of those before left out, so that their product stays within
    // a rounding of the power of exp(log_decay) (gradients of 26 tokens were off by 6.9e-7 with one rounded decay
    // and are by 1.5e-7 now).
    const Decay dec = decay_over(decay_log2(p.log_decay[h]), 1);
    float off = 0.f;
    // NaN under a decay that is NaN, which the first token in reverse would not show otherwise
    const float au = R.alpha_u_man * pow2i(R.alpha_u_exp) + (n > 0 ? 0.f * dec.m : 0.f);
    E* const out = static_cast<E*>(R.out) + token0 * R.ldo + h * D + col;
    E* to = out + (rev ? (n - 1) * R.ldo : 0);
    const long long step = rev ? -R.ldo : R.ldo;

    for (int tile = 0; tile < tiles; ++tile) {
        cp_async_wait<STAGES - 2>();
        const uint32_t raw = base + tile % STAGES * L::kTile;
        uint32_t at = raw;
        if constexpr (sizeof(E) == 2) {   // each thread widens the pieces that it copied
            at = base + STAGES * L::kTile + (tile & 1) * L::kWide;
#pragma unroll
            for (int q = 0; q < 3 * TT * L::kPerRow; q += D) {
                const int piece = q + col;   // the tensors' pieces follow one another
                uint32_t v[4];
                asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];"
                             : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3])
                             : "r"(raw + piece * 16));
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    const float2 x = pair_to_f(v[2 * half], E{}), y = pair_to_f(v[2 * half + 1], E{});
                    asm volatile("st.shared.v4.f32 [%0], {%1,%2,%3,%4};" ::"r"(at + piece * 32 + 16 * half), "f"(x.x),
                                 "f"(x.y), "f"(y.x), "f"(y.y)
                                 : "memory");
                }
            }
        }
        meet();   // the tile is there for all of the stream's threads, and the one before is done with
        if (tile + STAGES - 1 < tiles) load(tile + STAGES - 1);
        cp_async_commit();
        const int last = min(TT, steps - TT * tile);
        const float* rows = reinterpret_cast<const float*>(smem + (at - smem_u32(smem)));
#pragma unroll UNROLL
        for (int r = 0; r < TT; ++r) {
            if (r % UNROLL == 0 && r >= last) break;   // tokens past the last are zeros
            const int i = TT * tile + r;
            const float4* a = reinterpret_cast<const float4*>(rows + r * D);
            const float4* k = a + TT * D / 4;
            float g = 1.f;
            if (i < n && !(rev && i == 0)) {
                g = dec.c + (dec.m - off);
                off += (g - dec.c) - dec.m;
            }
            const float2 f = both(g), u = both(au * rows[2 * TT * D + r * D + col]);
            float2 sum[2] = {both(0.f), both(0.f)};
#pragma unroll
            for (int j = 0; j < D / 4; ++j) {
                const float4 av = a[j], bv = k[j];
                X[2 * j] = fma2(make_float2(bv.x, bv.y), u, mul2(X[2 * j], f));
                X[2 * j + 1] = fma2(make_float2(bv.z, bv.w), u, mul2(X[2 * j + 1], f));
                sum[0] = fma2(make_float2(av.x, av.y), X[2 * j], sum[0]);
                sum[1] = fma2(make_float2(av.z, av.w), X[2 * j + 1], sum[1]);
            }
            sum[0] = add2(sum[0], sum[1]);
            if (i < n) *to = from_f<E>(R.alpha_o * (sum[0].x + sum[0].y));
            to += step;
        }
    }
    if (!on) return;
    if (R.x_out) {
        const float2 f = both(rev && n > 0 ? dec.c + (dec.m - off) : 1.f);
        float* x = R.x_out + mat + (R.transposed ? col * D : col);
#pragma unroll
        for (int i = 0; i < D / 2; i += 2) {
            const float2 v = mul2(X[i], f), w = mul2(X[i + 1], f);
            if (R.transposed) {
                *reinterpret_cast<float4*>(x + 2 * i) = make_float4(v.x, v.y, w.x, w.y);
            } else {
                x[2 * i * D] = v.x;
                x[(2 * i + 1) * D] = v.y;
                x[(2 * i + 2) * D] = w.x;
                x[(2 * i + 3) * D] = w.y;
            }
        }
    }
    for (long long t = n; t < p.T; ++t) out[t * R.ldo] = from_f<E>(0.f);   // rows past the sequence's length
}

template <typename E, int D>
int launch_scan(int roles, const LinParams& p, cudaStream_t st)
{
    using L = ScanTile<E, D>;
    static_assert(L::kSmem <= 48 * 1024, "shared memory without an attribute");
    const long long blocks = (static_cast<long long>(p.B) * p.H + L::kStreams - 1) / L::kStreams;
    linattn_scan_kernel<E, D><<<dim3(static_cast<unsigned>(blocks), roles), kThreads, L::kSmem, st>>>(p);
    return launched();
}

template <typename E>
int by_width(int d, int roles, const LinParams& p, cudaStream_t st)
{
    if (d == 16) return launch_scan<E, 16>(roles, p, st);
    if (d == 32) return launch_scan<E, 32>(roles, p, st);
    return launch_scan<E, 64>(roles, p, st);
}

}  // namespace

bool linattn_scan_takes(int dtype, int d, int roles, const LinParams& p)
{
    // This kernel's time grows with every token, the chunked ones' with every chunk of d (or 128).  Where the GPU
    // holds all of the chunked kernel's CTAs at once, a chunk's latency is what they cost; beyond that a whole chunk's
    // work for each stream.  Measured (us, this kernel and the chunked ones): fp32, 2048 streams, d = 16: 6.4 and 8.1
    // at T = 26, 11.7 and 11.6 at 64; gradients at d = 64: 59 and 168 at 10, 146 and 172 at 40, 219 and 176 at 64;
    // bf16 gradients at d = 64: 77 and 111 at 16, 110 and 111 at 26, 152 and 111 at 40; 32 streams, fp32, d = 16: 3.4
    // and 3.4 at 10, 5.4 and 3.9 at 26; d = 64: 8.0 and 7.9 at 26; bf16, d = 16: 3.4 and 3.5 at 4, 4.0 and 3.4 at 10;
    // d = 64: 6.4 and 6.4 at 16, 8.6 and 6.5 at 26.
    const bool many = static_cast<long long>(p.B) * p.H * roles > 152LL * (d == 64 ? 2 : d == 32 ? 4 : 10);
    if (dtype == SRWM_F32) return p.T <= (many ? 40 : d == 64 ? 26 : 10);
    return p.T <= (many ? 20 : d / 4);
}

int linattn_scan_launch(int dtype, int d, int roles, const LinParams& p, cudaStream_t st)
{
    if (dtype == SRWM_F32) return by_width<float>(d, roles, p, st);
    if (dtype == SRWM_BF16) return by_width<__nv_bfloat16>(d, roles, p, st);
    return by_width<__half>(d, roles, p, st);
}

}  // namespace srwm
