// srwm_linattn_tc.cu -- the primitive of srwm_linattn.h on the 5th-generation
// tensor cores, for bf16 and d = 64: TMA tile loads and stores, tcgen05.mma
// with accumulators in tensor memory, one persistent CTA per SM.
//
// A chunk is 128 tokens, in their natural order whichever way the recurrence
// runs; in reverse the chunks are taken from the last one and the mask is the
// upper triangle.  With i, j in the chunk, nc its valid tokens, g the decay:
//   OX_i = alpha_u sum_j g^|i-j| (a_i . b_j) c_j         over the causal side
//   OI_i = a_i X,  out_i = alpha_o (g^e(i) OI_i + OX_i)   e = i + 1, or nc - 1 - i in reverse
//   U    = sum_j (w_j b_j) c_j^T,  X <- g^nc X + U        w_j = alpha_u g^(nc-1-j), or alpha_u g^(j+1)
// Five products per chunk: P = a b^T (128 x 128 x 64), OX (P from tensor
// memory, 128 x 64 x 128), OI (128 x 64 x 64), U (64 x 64 x 128).  a, b, c are
// the bf16 inputs themselves.  P and X enter their products as bf16 (high, low)
// pairs (2^-16), w_j b_j as three bf16 terms (2^-24), so that X, which is kept in
// fp32 registers, is good to fp32.  P as one bf16 took 63.7 instead of 67.3 us for the
// prompt below and 150 instead of 162 for its gradients, for a relative error of
// 0.00185 instead of the 0.00166 that the outputs' own rounding leaves.
//
// Warps: 0-7 turn P into its pair (one row per thread); 8-11 write the weighted b's
// terms; 12-15 hold X, add U to it and leave its pair in shared memory; 16-19
// write the outputs; 20 issues the TMA loads (three stages of a, b, c), 21 and 22
// the products.  Every stage of a chunk's work runs beside other stages of the
// same or the next chunk: P and X's chain meet only at the output.  Invalid
// tokens of a ragged chunk are zeroed in shared memory by warps 8-11 before
// anything reads them; past the tensor's end TMA fills zeros.  Every wait is
// bounded; a timeout sets the status word and ends the CTA after its copies and
// products in flight.
//
// What bounds it: 512 streams of 1024 tokens (268 MB in and out) take 64.6 us,
// 4.3 TB/s or 0.63 of the copy rate, their gradients 159 us; the chunked
// mma.sync kernel (srwm_linattn.cuh) takes 105 and 281 us.  A full chunk takes
// 1.55 us: the products keep the tensor pipe 47 % busy, and the six kinds of
// warps' loops share the instruction cache (their fetches at 54 % of its rate),
// which is why they are rolled and the waits' slow part is out of line.  512
// streams on 152 SMs also leave the last of four rounds a third full.
#include <atomic>

#include "srwm_check.h"
#include "srwm_ffgemm.h"
#include "srwm_linattn_tc.cuh"

namespace srwm {
namespace {

using namespace tc;

constexpr int STAGES = 3;
constexpr int kTileBytes = C * D * 2;
constexpr int kThreads = 736;
// First warps of the roles after the scores' eight; those that read tensor memory start at multiples of four, whose
// lanes they own in order.
constexpr int kTermWarp = 8, kStateWarp = 12, kOutWarp = 16, kLoadWarp = 20, kScoreMmaWarp = 21,
              kStateMmaWarp = 22;

// Tensor memory columns: P of two chunks, OI of two chunks, OX, U.  P's pair
// goes over it: 16 columns of fp32 become 8 of high and 8 of low halves.
constexpr uint32_t kP = 0, kOI = 256, kOX = 384, kU = 448, kTmemCols = 512;

struct TcMaps {
    CUtensorMap a, b, c, out;
};
struct TcParams {
    TcMaps map[3];
    LinParams lin;
    int roles, items;
    unsigned* status;
    unsigned long long wait_limit_ns;
    int skip_chunk;   // fault injection: where the loads of a stream end (-1: nowhere)
};

struct __align__(1024) Smem {
    uint8_t stage[STAGES][3][kTileBytes];   // a | b | c
    uint8_t terms[3][kTileBytes];           // of w_j b_j
    uint8_t state[2][D * D * 2];            // X's pair
    uint8_t out[4][32 * D * 2];             // per output warp: 32 rows
    float decay[8][64];                     // per score warp: g^|column - row| of a diagonal block, by their difference
    // A barrier's next phase never completes before every waiter of this one has passed, nor does an arrival for
    // it come before this one completes: where a producer may run a chunk ahead of a waiter or of another
    // producer, there are two of them, or one for each stage.
    uint64_t full[STAGES], empty[STAGES];
    uint64_t terms_full[2], terms_free[2];  // of a chunk's first and second 64 tokens
    uint64_t u_full, u_free, x_full, x_free, p32_full[2], p16_full[2], o_full[2], o_free[2], clean[STAGES];
    uint32_t tmem_base;
    int abort;
};

__global__ void __launch_bounds__(kThreads, 1) linattn_tc_kernel(const __grid_constant__ TcParams p)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem& sm = *reinterpret_cast<Smem*>(smem_raw);
    if ((smem_u32(smem_raw) & 1023u) != 0) {   // the swizzled tiles start on 1024-byte boundaries
        if (threadIdx.x == 0) atomicOr(p.status, kStatusSmemBase);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 2);
            mbar_init(&sm.clean[s], 4);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.terms_full[i], 4);
            mbar_init(&sm.terms_free[i], 1);
            mbar_init(&sm.p32_full[i], 1);
            mbar_init(&sm.p16_full[i], 8);
            mbar_init(&sm.o_full[i], 2);   // OX and OI, of which OI may be a chunk ahead
            mbar_init(&sm.o_free[i], 4);
        }
        mbar_init(&sm.u_full, 1);
        mbar_init(&sm.u_free, 4);
        mbar_init(&sm.x_full, 4);
        mbar_init(&sm.x_free, 1);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == kStateMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sm.tmem_base)),
                     "r"(kTmemCols)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    fence_before();
    __syncthreads();
    fence_after();
    const uint32_t tmem = sm.tmem_base;
    volatile int* abort = &sm.abort;
    // A warp's wait for phase `phase` of `bar`: the same answer for all of its lanes.
    auto wait = [&](uint64_t* bar, uint32_t phase) {
        return __all_sync(0xffffffffu, mbar_try_wait(bar, phase & 1u)) ||
               wait_slow(bar, phase & 1u, p.wait_limit_ns, abort, p.status);
    };
    // For two of them at once.
    auto wait2 = [&](uint64_t* bar, uint32_t phase, uint64_t* bar2, uint32_t phase2) {
        const bool here = mbar_try_wait(bar, phase & 1u), here2 = mbar_try_wait(bar2, phase2 & 1u);
        return __all_sync(0xffffffffu, here && here2) ||
               (wait_slow(bar, phase & 1u, p.wait_limit_ns, abort, p.status) &&
                wait_slow(bar2, phase2 & 1u, p.wait_limit_ns, abort, p.status));
    };
    // One arrival for the warp after its lanes' work.
    auto arrive = [&](uint64_t* bar) {
        __syncwarp();
        if (lane == 0) mbar_arrive(bar);
    };
    const uint32_t quad = static_cast<uint32_t>(32 * (warp & 3)) << 16;   // the warp's tensor memory lanes
    uint32_t g = 0;   // chunks so far, the same count in every warp

    if (warp == kLoadWarp) {
        // ---- loads
        if (lane == 0) {
            Walk<TcParams> w(p);
            for (; w.skip_empty() && !*abort; ++w.k, ++g) {
                const int s = g % STAGES;
                if (w.k == p.skip_chunk ||
                    !wait_bounded(&sm.empty[s], (g / STAGES + 1) & 1u, p.wait_limit_ns, abort, p.status))
                    break;
                const TcMaps& m = p.map[w.role];
                mbar_arrive_expect_tx(&sm.full[s], 3 * kTileBytes);
                tma_load_4d(sm.stage[s][1], &m.b, &sm.full[s], 0, w.h, w.token(), w.b);
                tma_load_4d(sm.stage[s][0], &m.a, &sm.full[s], 0, w.h, w.token(), w.b);
                tma_load_4d(sm.stage[s][2], &m.c, &sm.full[s], 0, w.h, w.token(), w.b);
            }
            drain_loads(sm.full, g);
        }
        __syncwarp();
    } else if (warp >= kScoreMmaWarp) {
        // ---- products: one warp issues P and OX, another U and OI, so that neither chain waits behind the other.
        // The whole warp walks the chunks, which keeps the descriptors in uniform registers; an elected lane issues.
        constexpr uint32_t id_p = idesc(true, C, C, false, false), id_u = idesc(true, D, D, true, true),
                           id_o = idesc(true, C, D, false, true);
        constexpr uint64_t kStage = 3 * kTileBytes / 16, kTile = kTileBytes / 16;   // descriptor steps
        const uint64_t d_stage = desc128(smem_u32(sm.stage[0][0]));
        bool ok = true;
        Walk<TcParams> w(p);
        if (warp == kScoreMmaWarp) {
            // P of chunk `at`, once its tiles have landed and been cleaned where they need it.  Its place was last
            // read by the product OX of chunk at - 2, issued before by this lane: products run in order.
            auto score = [&](uint32_t at) {
                if (!(ok = wait(&sm.full[at % STAGES], at / STAGES) &&
                           (!w.dirty() || wait(&sm.clean[at % STAGES], at / STAGES))))
                    return;
                fence_after();
                const uint64_t a = d_stage + kStage * (at % STAGES), b = a + kTile;
                const uint32_t to = tmem + kP + C * (at & 1);
                if (elect()) {
                    mma_ss<false>(to, a, b, id_p);
#pragma unroll
                    for (int k = 1; k < D / 16; ++k) mma_ss<true>(to, a + 2 * k, b + 2 * k, id_p);
                    commit(&sm.p32_full[at & 1]);
                }
                __syncwarp();
            };
            if (w.skip_empty()) score(0);
            for (; ok && w.skip_empty(); ++g) {
                const uint64_t c = d_stage + kStage * (g % STAGES) + 2 * kTile;
                ++w.k;
                if (w.skip_empty()) score(g + 1);   // the next chunk's, ahead of this one's output
                // the scores are there, and the outputs before have been read
                if (!ok || !(ok = wait2(&sm.p16_full[g & 1], g >> 1, &sm.o_free[(g - 1) & 1], (g - 1) >> 1))) break;
                fence_after();
                const uint32_t scores = tmem + kP + C * (g & 1);
                if (elect()) {
                    // low halves first, since each sum is cut off to fp32
                    mma_ts<false>(tmem + kOX, scores + 8, c, id_o);
#pragma unroll
                    for (int k = 1; k < 2 * C / 16; ++k)
                        mma_ts<true>(tmem + kOX, scores + 16 * (k % 8) + 8 * (k < 8), c + 128 * (k % 8), id_o);
                    commit(&sm.o_full[g & 1]);
                    commit(&sm.empty[g % STAGES]);
                }
                __syncwarp();
            }
        } else {
            const uint64_t d_terms = desc128(smem_u32(sm.terms[0])), d_state = desc128(smem_u32(sm.state[0]));
            for (; ok && w.skip_empty(); ++w.k, ++g) {
                const uint64_t a = d_stage + kStage * (g % STAGES), c = a + 2 * kTile;
                const uint32_t u = tmem + kU, oi = tmem + kOI + 64 * (g & 1);
                if (!(ok = wait2(&sm.full[g % STAGES], g / STAGES, &sm.u_free, g + 1))) break;
#pragma unroll
                for (int half = 0; half < 2; ++half) {
                    if (!(ok = wait(&sm.terms_full[half], g))) break;
                    fence_after();
                    if (elect()) {
                        const uint64_t t = d_terms + 512 * half, v = c + 512 * half;
                        // the small terms first, since each sum is cut off to fp32
                        if (half == 0)
                            mma_ss<false>(u, t + 2 * kTile, v, id_u);
                        else
                            mma_ss<true>(u, t + 2 * kTile, v, id_u);
#pragma unroll
                        for (int k = 1; k < 3 * 4; ++k)
                            mma_ss<true>(u, t + kTile * (2 - k / 4) + 128 * (k % 4), v + 128 * (k % 4), id_u);
                        commit(&sm.terms_free[half]);
                        if (half == 1) commit(&sm.u_full);
                    }
                    __syncwarp();
                }
                // X's copy is there, and the outputs that used this place have been read
                if (!ok || !(ok = wait2(&sm.x_full, g, &sm.o_free[g & 1], (g - 2) >> 1))) break;
                fence_after();
                if (elect()) {
                    mma_ss<false>(oi, a, d_state + 512, id_o);
#pragma unroll
                    for (int k = 1; k < 2 * D / 16; ++k)
                        mma_ss<true>(oi, a + 2 * (k % 4), d_state + 512 * (k < 4) + 128 * (k % 4), id_o);
                    commit(&sm.x_free);
                    commit(&sm.o_full[g & 1]);
                    commit(&sm.empty[g % STAGES]);
                }
                __syncwarp();
            }
        }
    } else if (warp < kTermWarp) {
        // ---- P as a pair, one row per thread; two sets of four warps take the 32-column blocks in turn
        const int own = warp & 3, set = warp >> 2, row = 32 * own + lane;
        float* decay = sm.decay[warp];
        bool ok = true;
        Walk<TcParams> w(p);
        for (; ok && !w.done(); w.next_item()) {
            const LinRole& R = p.lin.role[w.role];
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            const float au = R.alpha_u_man * pow2i(R.alpha_u_exp);
            // tab[x - l]: alpha_u g^|x - l| for row l, column x on the causal side of a diagonal block, 0 on the
            // other.  A block beside the diagonal takes the row's factor off: its columns are those of row 31 in
            // order, of row 0 in reverse.
            float* tab = decay + 31;
            __syncwarp();   // the table of the item before is no longer read
            for (int i = lane; i < 63; i += 32) {
                const int gap = w.rev ? i - 31 : 31 - i;
                tab[i - 31] = gap >= 0 ? au * exp2f(lg * static_cast<float>(gap)) : 0.f;
            }
            __syncwarp();
            const float* beside = w.rev ? tab : tab - 31;
            const int c0 = w.rev ? own : 0, c1 = w.rev ? 3 : own;
            const int first = c0 + ((c0 ^ set) & 1);   // this set's first block on the causal side
            for (; w.k < w.chunks; ++w.k, ++g) {
                if (!(ok = wait(&sm.p32_full[g & 1], g >> 1))) break;
                fence_after();
                const uint32_t P = tmem + quad + kP + C * (g & 1);
                for (int cb = set; cb < 4; cb += 2)   // the side that is masked
                    if (cb < c0 || cb > c1) {
                        const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                        for (int k = 0; k < 4; ++k) tmem_store8(P + 32 * cb + 8 * k, zero);
                    }
#pragma unroll 1
                for (int hb = 2 * first; hb <= 2 * c1 + 1; hb += (hb & 1) ? 3 : 1) {   // 16 columns of this set's blocks
                    const int cb = hb >> 1, x0 = 16 * (hb & 1);
                    uint32_t r[16], hi[8], lo[8];
                    tmem_rows(P + 16 * hb, r);
                    const int beyond = w.rev ? 32 * cb - row : row - 32 * cb - 31;
                    const float f = exp2f(lg * static_cast<float>(max(0, beyond)));
                    const float* col = (cb == own ? tab - lane : beside) + x0;
                    tmem_wait(r);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 w = mul2(both(f), make_float2(col[2 * k], col[2 * k + 1]));
                        float2 v = mul2(as_float2(r[2 * k], r[2 * k + 1]), w);
                        hi[k] = take_bf16(v);
                        lo[k] = pack_bf16(v);
                    }
                    tmem_store8(P + 16 * hb, hi);
                    tmem_store8(P + 16 * hb + 8, lo);
                }
                tmem_store_wait();
                fence_before();
                arrive(&sm.p16_full[g & 1]);
            }
        }
    } else if (warp < kStateWarp) {
        // ---- the terms of w_j b_j: 64 tokens at a time, so that the products of one half run while the other is
        // written; half a token's row per thread
        const int t = threadIdx.x - 32 * kTermWarp, q0 = t >> 6 << 2;
        bool ok = true;
        Walk<TcParams> w(p);
        for (; ok && !w.done(); w.next_item()) {
            const LinRole& R = p.lin.role[w.role];
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            const float au = R.alpha_u_man * pow2i(R.alpha_u_exp);
            for (; ok && w.k < w.chunks; ++w.k, ++g) {
                const int s = g % STAGES, nc = w.valid();
                if (!(ok = wait(&sm.full[s], g / STAGES))) break;
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    const int j = 64 * half + (t & 63);
                    const float wj = au * exp2f(lg * static_cast<float>(w.rev ? j + 1 : max(0, nc - 1 - j)));
                    if (!(ok = wait(&sm.terms_free[half], g + 1))) break;   // those of the chunk before have been read
                    const uint32_t at = smem_u32(sm.stage[s][1]) + 128 * j, to = smem_u32(sm.terms[0]) + 128 * j;
                    const bool clean = j >= nc && w.dirty();
                    const uint32_t zero[4] = {0, 0, 0, 0};
                    uint32_t ahead[4];
                    lds128(at + static_cast<uint32_t>((q0 ^ (j & 7)) << 4), ahead);
#pragma unroll 1
                    for (int q = q0; q < q0 + 4; ++q) {
                        const uint32_t o = static_cast<uint32_t>((q ^ (j & 7)) << 4);
                        uint32_t t0[4], t1[4], t2[4];
                        float2 v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) v[k] = mul2(unpack_bf16(clean ? 0 : ahead[k]), both(wj));
                        lds128(at + static_cast<uint32_t>((((q + 1) & 7) ^ (j & 7)) << 4), ahead);
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            t0[k] = take_bf16(v[k]);
                            t1[k] = take_bf16(v[k]);
                            t2[k] = pack_bf16(v[k]);
                        }
                        sts128(to + o, t0);
                        sts128(to + o + kTileBytes, t1);
                        sts128(to + o + 2 * kTileBytes, t2);
                        if (clean) {
                            sts128(at + o, zero);
                            sts128(at + o - kTileBytes, zero);   // a's and c's tiles lie on either side
                            sts128(at + o + kTileBytes, zero);
                        }
                    }
                    fence_proxy_async_smem();
                    if (half == 1) arrive(&sm.clean[s]);   // first: this phase ends before the stage is given up
                    arrive(&sm.terms_full[half]);
                }
            }
        }
    } else if (warp < kOutWarp) {
        // ---- the state
        const int own = warp - kStateWarp, r4 = lane >> 2, x2 = 2 * (lane & 3);
        bool ok = true;
        Walk<TcParams> w(p);
        for (; ok && !w.done(); w.next_item()) {
            const LinRole& R = p.lin.role[w.role];
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            const size_t mat = (static_cast<size_t>(w.b) * p.lin.H + w.h) * D * D;
            float2 X[8][2];   // rows 16 own + r4 (+ 8), columns 8 t + x2 and the next
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = 16 * own + r4 + 8 * k, q = 8 * t + x2;
                    X[t][k] = !R.x_in       ? both(0.f)
                              : R.transposed ? make_float2(R.x_in[mat + q * D + i], R.x_in[mat + (q + 1) * D + i])
                                             : *reinterpret_cast<const float2*>(R.x_in + mat + i * D + q);
                }
            const Decay full = decay_over(lg, C);
            for (; w.k < w.chunks; ++w.k, ++g) {
                if (!(ok = wait(&sm.x_free, g + 1))) break;
#pragma unroll
                for (int t = 0; t < 8; ++t)   // X's pair
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        float2 v = X[t][k];
                        const uint32_t to = state_at<D>(smem_u32(sm.state[0]), 16 * own + r4 + 8 * k, t, 0) + 2 * x2;
                        const uint32_t hi = take_bf16(v), lo = pack_bf16(v);
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(hi) : "memory");
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + D * D * 2), "r"(lo) : "memory");
                    }
                fence_proxy_async_smem();
                arrive(&sm.x_full);
                const int nc = w.valid();
                if (!(ok = wait(&sm.u_full, g))) break;
                fence_after();
                {
                    const Decay dec = nc == C ? full : decay_over(lg, nc);
#pragma unroll
                    for (int part = 0; part < 2; ++part) {
                        uint32_t u[16];
                        tmem_frag32(tmem + quad + kU + 32 * part, u);
                        tmem_wait(u);
#pragma unroll
                        for (int t = 0; t < 4; ++t)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float2& x = X[4 * part + t][k];
                                const float2 add = as_float2(u[4 * t + 2 * k], u[4 * t + 2 * k + 1]);
                                x = fma2(x, both(dec.m), fma2(x, both(dec.c), add));
                            }
                    }
                    fence_before();
                    arrive(&sm.u_free);
                }
            }
            if (ok && R.x_out)
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const int i = 16 * own + r4 + 8 * k, q = 8 * t + x2;
                        R.x_out[mat + (R.transposed ? q * D + i : i * D + q)] = X[t][k].x;
                        R.x_out[mat + (R.transposed ? (q + 1) * D + i : i * D + q + 1)] = X[t][k].y;
                    }
        }
    } else if (warp < kLoadWarp) {
        // ---- the outputs, one row per thread
        const int own = warp - kOutWarp;
        bool ok = true;
        Walk<TcParams> w(p);
        for (; ok && !w.done(); w.next_item()) {
            const LinRole& R = p.lin.role[w.role];
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            for (; w.k < w.chunks; ++w.k, ++g) {
                const int nc = w.valid();
                if (!(ok = wait(&sm.o_full[g & 1], g >> 1))) break;
                fence_after();
                const int i = 32 * own + lane;
                const float alpha = R.alpha_o;
                const float f = alpha * exp2f(lg * static_cast<float>(w.rev ? max(0, nc - 1 - i) : i + 1));
                if (lane == 0) bulk_wait_read<0>();   // the rows before have left the staging buffer
                __syncwarp();
#pragma unroll 1
                for (int part = 0; part < 4; ++part) {
                    uint32_t oi[16], ox[16];
                    tmem_rows(tmem + quad + kOI + 64 * (g & 1) + 16 * part, oi);
                    tmem_rows(tmem + quad + kOX + 16 * part, ox);
                    tmem_wait(oi);
                    tmem_wait(ox);
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        uint32_t v[4];
#pragma unroll
                        for (int k = 0; k < 4; ++k) {
                            const int x = 8 * q + 2 * k;
                            v[k] = pack_bf16(fma2(as_float2(oi[x], oi[x + 1]), both(f),
                                                  mul2(both(alpha), as_float2(ox[x], ox[x + 1]))));
                            if (i >= nc) v[k] = 0;   // 0 times what is not finite
                        }
                        sts128(smem_u32(sm.out[own]) + 128 * lane + (((2 * part + q) ^ (lane & 7)) << 4), v);
                    }
                }
                fence_before();
                arrive(&sm.o_free[g & 1]);
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0 && w.token() + 32 * own < p.lin.T) {
                    tma_store_4d(&p.map[w.role].out, sm.out[own], 0, w.h, w.token() + 32 * own, w.b);
                    bulk_commit();
                }
            }
            // tokens past the last chunk
            __nv_bfloat16* po =
                static_cast<__nv_bfloat16*>(R.out) + static_cast<long long>(w.b) * p.lin.T * R.ldo + w.h * D;
            const long long z0 = static_cast<long long>(w.chunks) * C, pieces = (p.lin.T - z0) * (D / 8);
            for (long long q = threadIdx.x - 32 * kOutWarp; q < pieces; q += 128)
                *reinterpret_cast<uint4*>(po + (z0 + q / (D / 8)) * R.ldo + q % (D / 8) * 8) = make_uint4(0, 0, 0, 0);
        }
        if (lane == 0) bulk_wait_all<0>();   // the rows in flight are written before the CTA ends
        __syncwarp();
    }

    fence_before();
    __syncthreads();
    fence_after();
    if (warp == kStateMmaWarp) {
        if (*abort) let_products_end();
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
}

}  // namespace

// fp16 stays with the other kernel: its scores would have to enter as pairs, as in fp32.
bool linattn_tc_takes(int dtype, int d, const LinParams& p)
{
    return dtype != SRWM_F16 && d == D && p.segments == 1 && p.T >= C;
}

int linattn_tc_launch(int roles, const LinParams& lin, cudaStream_t st)
{
    TcParams p{};
    p.lin = lin;
    p.roles = roles;
    const long long items = static_cast<long long>(lin.B) * lin.H * roles;
    if (items > 0x7fffffffLL - 1024) return SRWM_ERR_SHAPE;
    p.items = static_cast<int>(items);
    int rc = device_status_ptr(&p.status);
    if (rc != SRWM_OK) return rc;
    p.wait_limit_ns = device_wait_limit_ns();
    p.skip_chunk = debug_skip_chunk();
    for (int i = 0; i < roles; ++i) {
        const LinRole& r = lin.role[i];
        if ((rc = token_map(&p.map[i].a, r.a, r.lda, lin, C, false)) != SRWM_OK ||
            (rc = token_map(&p.map[i].b, r.b, r.ldb, lin, C, false)) != SRWM_OK ||
            (rc = token_map(&p.map[i].c, r.c, r.ldc, lin, C, false)) != SRWM_OK ||
            (rc = token_map(&p.map[i].out, r.out, r.ldo, lin, 32, false)) != SRWM_OK)
            return rc;
    }
    static std::atomic<int> sms[kMaxDevices];   // 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    constexpr int smem = static_cast<int>(sizeof(Smem));
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    int n_sm = sms[dev].load();
    if (n_sm == 0) {
        if (cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(reinterpret_cast<const void*>(linattn_tc_kernel), cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 smem) != cudaSuccess) {
            cudaGetLastError();
            return SRWM_ERR_CUDA;
        }
        sms[dev].store(n_sm);
    }
    linattn_tc_kernel<<<p.items < n_sm ? p.items : n_sm, kThreads, smem, st>>>(p);
    return launched();
}

}  // namespace srwm
