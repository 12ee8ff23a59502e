// srwm_linattn_tc32.cu -- the primitive of srwm_linattn.h on the 5th-generation
// tensor cores, for fp32 and d = 64.  The chunk, its five products and the
// pipeline are those of srwm_linattn_tc.cu; what differs is the operands'
// precision.
//
// Every operand is a pair of fp16 values, x ~ (high + low) 2^e with one
// exponent for 16 tokens (22 bits of the largest of them, see
// srwm_linattn.cuh), and every product three: high high, high low, low high.
// a, b, c land as fp32 in two tiles of 32 columns each, and are turned into
// their pairs in place: a row's high halves take its 128 bytes of the first
// tile, the low halves those of the second.  The scores of 16 columns carry
// 2^(eb + ec) relative to the largest that their 16 rows see, the weighted b's
// terms relative to the chunk's largest, and X's copy the exponent of a bound
// on X; sums are fp32 throughout.
//
// Warps: 0-7 turn P into its pair; 8-11 write the weighted b's terms, 32 tokens
// at a time into two buffers in turn; 12-15 hold X; 16-19 convert c and write
// the outputs; 20-23 convert a and b; 24 issues the TMA loads (two stages), 25 and
// 26 the products.
//
// What bounds it: 128 streams of 8192 tokens (1.08 GB in and out) take 316 us,
// 0.50 of the copy rate; the chunked mma.sync kernel (srwm_linattn.cuh) takes
// 505 us split over the axis and 547 unsplit.  A chunk takes 4.6 us, of which
// its three products per product keep the tensor pipe 26 % busy and the
// conversions, the terms and the scores' pairs their warps: 41 % of the issue
// slots, with the instruction cache at 51 % of its rate.  Two stages of 96 KB
// leave no room for a third; a stage released tensor by tensor gained 1 % here
// and cost 8 % in gradients of 512 streams of 512 tokens, which take 217 us.
#include <atomic>

#include "srwm_check.h"
#include "srwm_ffgemm.h"
#include "srwm_linattn_tc.cuh"

namespace srwm {
namespace {

using namespace tc;

constexpr int STAGES = 2, RING = 4;
constexpr int kHalfTile = C * 128;   // bytes: 32 columns of fp32, or 64 of fp16
constexpr int kThreads = 864;
constexpr int kTermWarp = 8, kStateWarp = 12, kOutWarp = 16, kConvertWarp = 20, kLoadWarp = 24, kScoreMmaWarp = 25,
              kStateMmaWarp = 26;

// Tensor memory columns: P of two chunks, OI of two chunks, OX, U.  P's pair
// goes over it: 16 columns of fp32 become 8 of high and 8 of low halves.
constexpr uint32_t kP = 0, kOI = 256, kOX = 384, kU = 448, kTmemCols = 512;

struct Tc32Maps {
    CUtensorMap a, b, c;
};
struct Tc32Params {
    Tc32Maps map[3];
    LinParams lin;
    int roles, items;
    unsigned* status;
    unsigned long long wait_limit_ns;
    int skip_chunk;   // fault injection: where the loads of a stream end (-1: nowhere)
};

struct __align__(1024) Smem32 {
    uint8_t stage[STAGES][3][2][kHalfTile];   // a | b | c: columns 0-31 | 32-63, then high | low halves
    uint8_t terms[2][2][32 * 128];            // of w_j b_j for 32 tokens: high | low
    uint8_t state[2][D * D * 2];              // X's copy: high | low
    float decay[8][64];
    int exps[RING][3][8];                     // of a, b, c, per 16 tokens
    int norm[RING][9];                        // the exponents that normalise the scores of 16 rows each, and the terms
    int state_exp[RING];
    int valid[RING], total;                   // valid tokens of a chunk; chunks of this CTA
    float top[2][4];                          // largest |X| of each state warp's rows at an item's start
    uint64_t full[STAGES], empty[STAGES];
    uint64_t ready_ab[STAGES], ready_c[STAGES], norm_full[STAGES];   // the tiles are pairs, and norm is there
    uint64_t terms_full[2], terms_free[2];
    uint64_t u_full, u_free, x_full, x_free, p32_full[2], p16_full[2], o_full[2], o_free[2], top_full;
    uint32_t tmem_base;
    int abort;
};

// Sixteen tokens of a landed fp32 tile into pairs, in place, two lanes per
// token; tokens at and past nc become zeros.
__device__ __forceinline__ void convert_tokens(uint8_t* tiles, int group, int nc, int* exponent)
{
    const int lane = threadIdx.x & 31, half = lane & 1, r = 16 * group + (lane >> 1);
    const uint32_t tile = smem_u32(tiles) + 128 * r;
    const bool valid = r < nc;
    uint32_t v[8][4];   // piece k holds columns 4 (k ^ 4 half) .. of this lane's tile: its lanes' banks differ
    float m = 0.f;
#pragma unroll
    for (int k = 0; k < 8; ++k) {
        lds128(tile + half * kHalfTile + (((k ^ (half << 2)) ^ (r & 7)) << 4), v[k]);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            if (!valid) v[k][i] = 0;
            m = fmaxf(m, fabsf(__uint_as_float(v[k][i])));
        }
    }
    const uint32_t top = __reduce_max_sync(0xffffffffu, __float_as_uint(m));   // every lane has read its row
    const int ex = max(static_cast<int>(top >> 23), 14);                       // 2^(ex-127) <= top < 2^(ex-126)
    const float sc = __int_as_float((267 - ex) << 23);                         // top * sc in [2^13, 2^14)
    if (lane == 0) *exponent = top == 0 ? kNoValue : ex - 140;
    __syncwarp();
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        uint32_t hi[4], lo[4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
            split_half2_2(mul2(as_float2(v[2 * k + i / 2][i % 2 * 2], v[2 * k + i / 2][i % 2 * 2 + 1]), both(sc)), hi[i],
                          lo[i]);
        const uint32_t o = static_cast<uint32_t>(((4 * half + (k ^ (half << 1))) ^ (r & 7)) << 4);
        sts128(tile + o, hi);
        sts128(tile + o + kHalfTile, lo);
    }
}

__global__ void __launch_bounds__(kThreads, 1) linattn_tc32_kernel(const __grid_constant__ Tc32Params p)
{
    extern __shared__ __align__(1024) unsigned char smem_raw[];
    Smem32& sm = *reinterpret_cast<Smem32*>(smem_raw);
    if ((smem_u32(smem_raw) & 1023u) != 0) {   // the swizzled tiles start on 1024-byte boundaries
        if (threadIdx.x == 0) atomicOr(p.status, kStatusSmemBase);
        return;
    }
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 2);
            mbar_init(&sm.ready_ab[s], 4);
            mbar_init(&sm.ready_c[s], 4);
            mbar_init(&sm.norm_full[s], 4);
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
        mbar_init(&sm.top_full, 4);
        sm.abort = 0;
        fence_mbar_init();
    }
    if (warp == kLoadWarp) {
        int total = 0;
        for (int item = blockIdx.x + gridDim.x * lane; item < p.items; item += 32 * gridDim.x) {
            const int n = p.lin.lengths ? min(max(p.lin.lengths[item / p.roles / p.lin.H], 0), p.lin.T) : p.lin.T;
            total += (n + C - 1) / C;
        }
        total = __reduce_add_sync(0xffffffffu, total);
        if (lane == 0) sm.total = total;
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
            Walk<Tc32Params> w(p);
            for (; w.skip_empty() && !*abort; ++w.k, ++g) {
                const int s = g % STAGES;
                if (w.k == p.skip_chunk ||
                    !wait_bounded(&sm.empty[s], (g / STAGES + 1) & 1u, p.wait_limit_ns, abort, p.status))
                    break;
                const Tc32Maps& m = p.map[w.role];
                sm.valid[g % RING] = w.valid();
                mbar_arrive_expect_tx(&sm.full[s], 6 * kHalfTile);
#pragma unroll 1
                for (int half = 0; half < 2; ++half) {
                    tma_load_4d(sm.stage[s][1][half], &m.b, &sm.full[s], 32 * half, w.h, w.token(), w.b);
                    tma_load_4d(sm.stage[s][0][half], &m.a, &sm.full[s], 32 * half, w.h, w.token(), w.b);
                    tma_load_4d(sm.stage[s][2][half], &m.c, &sm.full[s], 32 * half, w.h, w.token(), w.b);
                }
            }
            drain_loads(sm.full, g);
        }
        __syncwarp();
    } else if (warp >= kScoreMmaWarp) {
        // ---- products: one warp issues P and OX, another U and OI.  The whole warp walks the chunks, which keeps
        // the descriptors in uniform registers; an elected lane issues.
        constexpr uint32_t id_p = idesc(false, C, C, false, false), id_u = idesc(false, D, D, true, true),
                           id_o = idesc(false, C, D, false, true);
        constexpr uint64_t kStage = 6 * kHalfTile / 16, kTile = 2 * kHalfTile / 16, kLow = kHalfTile / 16;
        const uint64_t d_stage = desc128(smem_u32(sm.stage[0][0][0]));
        bool ok = true;
        Walk<Tc32Params> w(p);
        if (warp == kScoreMmaWarp) {
            // P of chunk `at`, once a and b are pairs.  Its place was last read by the product OX of chunk at - 2,
            // issued before by this lane: products run in order.
            auto score = [&](uint32_t at) {
                if (!(ok = wait(&sm.ready_ab[at % STAGES], at / STAGES))) return;
                fence_after();
                const uint64_t a = d_stage + kStage * (at % STAGES), b = a + kTile;
                const uint32_t to = tmem + kP + C * (at & 1);
                if (elect()) {
                    // low high, high low, high high: the small products first, since each sum is cut off to fp32
                    mma_ss<false>(to, a + kLow, b, id_p);
#pragma unroll
                    for (int k = 1; k < 3 * 4; ++k)
                        mma_ss<true>(to, a + (k < 4) * kLow + 2 * (k % 4), b + (k / 4 == 1) * kLow + 2 * (k % 4), id_p);
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
                    mma_ts<false>(tmem + kOX, scores + 8, c, id_o);
#pragma unroll
                    for (int k = 1; k < 3 * 8; ++k)
                        mma_ts<true>(tmem + kOX, scores + 16 * (k % 8) + 8 * (k < 8),
                                     c + (k / 8 == 1) * kLow + 128 * (k % 8), id_o);
                    commit(&sm.o_full[g & 1]);
                    commit(&sm.empty[g % STAGES]);
                }
                __syncwarp();
            }
        } else {
            const uint64_t d_terms = desc128(smem_u32(sm.terms[0][0])), d_state = desc128(smem_u32(sm.state[0]));
            for (; ok && w.skip_empty(); ++w.k, ++g) {
                const uint64_t a = d_stage + kStage * (g % STAGES), c = a + 2 * kTile;
                const uint32_t u = tmem + kU, oi = tmem + kOI + 64 * (g & 1);
                if (!(ok = wait2(&sm.ready_ab[g % STAGES], g / STAGES, &sm.ready_c[g % STAGES], g / STAGES) &&
                           wait(&sm.u_free, g + 1)))
                    break;
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    if (!(ok = wait(&sm.terms_full[q & 1], 2 * g + (q >> 1)))) break;
                    fence_after();
                    if (elect()) {
                        const uint64_t t = d_terms + 512 * (q & 1), v = c + 256 * q;   // 32 tokens: 4 KB of a tile
                        if (q == 0)
                            mma_ss<false>(u, t + 256, v, id_u);
                        else
                            mma_ss<true>(u, t + 256, v, id_u);
#pragma unroll
                        for (int k = 1; k < 3 * 2; ++k)
                            mma_ss<true>(u, t + (k < 2) * 256 + 128 * (k % 2),
                                         v + (k / 2 == 1) * kLow + 128 * (k % 2), id_u);
                        commit(&sm.terms_free[q & 1]);
                        if (q == 3) commit(&sm.u_full);
                    }
                    __syncwarp();
                }
                // X's copy is there, and the outputs that used this place have been read
                if (!ok || !(ok = wait2(&sm.x_full, g, &sm.o_free[g & 1], (g - 2) >> 1))) break;
                fence_after();
                if (elect()) {
                    mma_ss<false>(oi, a + kLow, d_state, id_o);
#pragma unroll
                    for (int k = 1; k < 3 * 4; ++k)
                        mma_ss<true>(oi, a + (k < 4) * kLow + 2 * (k % 4),
                                     d_state + 512 * (k / 4 == 1) + 128 * (k % 4), id_o);
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
        bool ok = true;
        Walk<Tc32Params> w(p);
        for (; ok && !w.done(); w.next_item()) {
            const LinRole& R = p.lin.role[w.role];
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            // tab[x - l]: alpha_u's mantissa times g^|x - l| for row l, column x on the causal side of a diagonal
            // block, 0 on the other.  A block beside the diagonal takes the row's factor off: its columns are those
            // of row 31 in order, of row 0 in reverse.
            float* tab = sm.decay[warp] + 31;
            __syncwarp();   // the table of the item before is no longer read
            for (int i = lane; i < 63; i += 32) {
                const int gap = w.rev ? i - 31 : 31 - i;
                tab[i - 31] = gap >= 0 ? R.alpha_u_man * exp2f(lg * static_cast<float>(gap)) : 0.f;
            }
            __syncwarp();
            const float* beside = w.rev ? tab : tab - 31;
            const int c0 = w.rev ? own : 0, c1 = w.rev ? 3 : own;
            const int first = c0 + ((c0 ^ set) & 1);   // this set's first block on the causal side
            for (; w.k < w.chunks; ++w.k, ++g) {
                if (!(ok = wait2(&sm.p32_full[g & 1], g >> 1, &sm.norm_full[g % STAGES], g / STAGES))) break;
                fence_after();
                const int(&e)[3][8] = sm.exps[g % RING];
                const int ef = sm.norm[g % RING][row >> 4] + 20;
                const uint32_t P = tmem + quad + kP + C * (g & 1);
                for (int cb = set; cb < 4; cb += 2)   // the side that is masked
                    if (cb < c0 || cb > c1) {
                        const uint32_t zero[8] = {0, 0, 0, 0, 0, 0, 0, 0};
#pragma unroll
                        for (int k = 0; k < 4; ++k) tmem_store8(P + 32 * cb + 8 * k, zero);
                    }
#pragma unroll 1
                for (int hb = 2 * first; hb <= 2 * c1 + 1; hb += (hb & 1) ? 3 : 1) {   // 16 columns of this set's blocks
                    const int cb = hb >> 1;
                    uint32_t r[16], hi[8], lo[8];
                    tmem_rows(P + 16 * hb, r);
                    const int beyond = w.rev ? 32 * cb - row : row - 32 * cb - 31;
                    const float f = exp2f(lg * static_cast<float>(max(0, beyond))) * pow2i(e[1][hb] + e[2][hb] - ef);
                    const float* col = (cb == own ? tab - lane : beside) + 16 * (hb & 1);
                    tmem_wait(r);
#pragma unroll
                    for (int k = 0; k < 8; ++k) {
                        const float2 w2 = mul2(both(f), make_float2(col[2 * k], col[2 * k + 1]));
                        split_half2_2(mul2(as_float2(r[2 * k], r[2 * k + 1]), w2), hi[k], lo[k]);
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
        // ---- the terms of w_j b_j, 32 tokens at a time: one token per lane, 16 columns per warp
        const int own = warp - kTermWarp;
        bool ok = true;
        Walk<Tc32Params> w(p);
        for (; ok && !w.done(); w.next_item()) {
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            for (; ok && w.k < w.chunks; ++w.k, ++g) {
                const int s = g % STAGES, nc = w.valid();
                if (!(ok = wait2(&sm.ready_ab[s], g / STAGES, &sm.ready_c[s], g / STAGES))) break;
                const int(&e)[3][8] = sm.exps[g % RING];
                // The largest 2^(eb + ec) g^gap among the column groups on the causal side of 16 rows (lanes 0-7 the
                // first of this warp's, 8-15 the others: a group that no row sees must not cost them their bits), and
                // among all with their distance to the chunk's end: what the scores and the terms are relative to.
                int eu;
                {
                    const int c = lane & 7, strip = 2 * own + ((lane >> 3) & 1), r0 = 16 * strip;
                    const float ec = static_cast<float>(e[1][c] + e[2][c]);
                    const int gap = w.rev ? 16 * c - r0 - 15 : r0 - 16 * c - 15;
                    const int end = w.rev ? 16 * c + 1 : max(0, nc - 16 * c - 16);
                    const bool causal = w.rev ? c >= strip : c <= strip;
                    float top = causal ? fmaf(lg, static_cast<float>(max(0, gap)), ec) : -8000.f;
                    float last = fmaf(lg, static_cast<float>(end), ec);
#pragma unroll
                    for (int o = 4; o > 0; o >>= 1) {
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
                        last = fmaxf(last, __shfl_xor_sync(0xffffffffu, last, o));
                    }
                    eu = static_cast<int>(ceilf(fmaxf(last, -8000.f)));
                    if (lane < 16 && c == 0) sm.norm[g % RING][strip] = static_cast<int>(ceilf(fmaxf(top, -8000.f)));
                    if (own == 0 && lane == 0) sm.norm[g % RING][8] = eu;
                    arrive(&sm.norm_full[s]);
                }
#pragma unroll 1
                for (int q = 0; q < 4; ++q) {
                    const int j = 32 * q + lane;
                    const float wj = exp2f(lg * static_cast<float>(w.rev ? j + 1 : max(0, nc - 1 - j))) *
                                     pow2i(e[1][j >> 4] + e[2][j >> 4] - eu);
                    if (!(ok = wait(&sm.terms_free[q & 1], 2 * g + (q >> 1) + 1))) break;   // those before have been read
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        const uint32_t o = static_cast<uint32_t>(((2 * own + i) ^ (j & 7)) << 4);
                        const uint32_t from = smem_u32(sm.stage[s][1][0]) + 128 * j + o;
                        const uint32_t to = smem_u32(sm.terms[q & 1][0]) + 128 * lane + o;
                        uint32_t h[4], l[4];
                        lds128(from, h);
                        lds128(from + kHalfTile, l);
#pragma unroll
                        for (int k = 0; k < 4; ++k)
                            split_half2_2(mul2(add2(unpack_half2(h[k]), unpack_half2(l[k])), both(wj)), h[k], l[k]);
                        sts128(to, h);
                        sts128(to + 32 * 128, l);
                    }
                    fence_proxy_async_smem();
                    arrive(&sm.terms_full[q & 1]);
                }
            }
        }
    } else if (warp < kOutWarp) {
        // ---- the state
        const int own = warp - kStateWarp, r4 = lane >> 2, x2 = 2 * (lane & 3);
        uint32_t starts = 0;   // items that began with a state
        bool ok = true;
        Walk<Tc32Params> w(p);
        for (; ok && !w.done(); w.next_item()) {
            const LinRole& R = p.lin.role[w.role];
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            const size_t mat = (static_cast<size_t>(w.b) * p.lin.H + w.h) * D * D;
            float2 X[8][2];   // rows 16 own + r4 (+ 8), columns 8 t + x2 and the next
            float bound = 0.f;   // >= every |X|, the same in every state warp
#pragma unroll
            for (int t = 0; t < 8; ++t)
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int i = 16 * own + r4 + 8 * k, q = 8 * t + x2;
                    X[t][k] = !R.x_in       ? both(0.f)
                              : R.transposed ? make_float2(R.x_in[mat + q * D + i], R.x_in[mat + (q + 1) * D + i])
                                             : *reinterpret_cast<const float2*>(R.x_in + mat + i * D + q);
                    bound = fmaxf(bound, fmaxf(fabsf(X[t][k].x), fabsf(X[t][k].y)));
                }
            if (R.x_in && w.chunks > 0) {
                bound = __uint_as_float(__reduce_max_sync(0xffffffffu, __float_as_uint(bound)));
                if (lane == 0) sm.top[starts & 1][own] = bound;
                arrive(&sm.top_full);
                if (!(ok = wait(&sm.top_full, starts))) break;
                for (int i = 0; i < 4; ++i) bound = fmaxf(bound, sm.top[starts & 1][i]);
                ++starts;
            }
            const Decay full = decay_over(lg, C);
            for (; w.k < w.chunks; ++w.k, ++g) {
                if (!(ok = wait(&sm.x_free, g + 1))) break;
                const int eb = max(static_cast<int>(__float_as_uint(bound) >> 23), 14);
                const float sc = bound == 0.f ? 0.f : pow2i(140 - eb);   // X's copy: X * 2^-(eb - 140), at most 2^14
                if (own == 0 && lane == 0) sm.state_exp[g % RING] = bound == 0.f ? kNoValue : eb - 140;
#pragma unroll
                for (int t = 0; t < 8; ++t)
#pragma unroll
                    for (int k = 0; k < 2; ++k) {
                        const uint32_t to = state_at<D>(smem_u32(sm.state[0]), 16 * own + r4 + 8 * k, t, 0) + 2 * x2;
                        uint32_t hi, lo;
                        split_half2_2(mul2(X[t][k], both(sc)), hi, lo);
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(hi) : "memory");
                        asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + D * D * 2), "r"(lo) : "memory");
                    }
                fence_proxy_async_smem();
                arrive(&sm.x_full);
                const int nc = w.valid();
                if (!(ok = wait(&sm.u_full, g))) break;
                fence_after();
                const int eu = sm.norm[g % RING][8] + R.alpha_u_exp;
                // X = g^nc X + alpha_u U 2^eu, in two factors that stay inside fp32's range
                const float f1 = pow2i(eu / 2), f2 = R.alpha_u_man * pow2i(eu - eu / 2);
                const Decay dec = nc == C ? full : decay_over(lg, nc);
#pragma unroll
                for (int part = 0; part < 4; ++part) {
                    uint32_t u[8];
                    tmem_frag16(tmem + quad + kU + 16 * part, u);
                    tmem_wait(u);
#pragma unroll
                    for (int t = 0; t < 2; ++t)
#pragma unroll
                        for (int k = 0; k < 2; ++k) {
                            float2& x = X[2 * part + t][k];
                            x = fma2(mul2(as_float2(u[4 * t + 2 * k], u[4 * t + 2 * k + 1]), both(f1)), both(f2),
                                     fma2(x, both(dec.m), mul2(x, both(dec.c))));
                        }
                }
                fence_before();
                arrive(&sm.u_free);
                // |U| < C 2^28
                const float most = fabsf(f2) * static_cast<float>(C) * pow2i(28 + eu / 2);
                bound = fminf(fmaf(bound, dec.m + dec.c, most) * 1.0001f, 1.7e38f);
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
    } else if (warp < kConvertWarp) {
        // ---- the outputs, one row per thread, written from registers; and the next chunk's c into pairs before
        // this one's outputs are there
        const int own = warp - kOutWarp, i = 32 * own + lane;
        Walk<Tc32Params> w(p);
        auto convert = [&](uint32_t at) {
            const int s = at % STAGES;
            if (!wait(&sm.full[s], at / STAGES)) return false;
#pragma unroll 1
            for (int group = 2 * own; group < 2 * own + 2; ++group)
                convert_tokens(sm.stage[s][2][0], group, sm.valid[at % RING], &sm.exps[at % RING][2][group]);
            fence_proxy_async_smem();
            arrive(&sm.ready_c[s]);
            return true;
        };
        bool ok = sm.total == 0 || convert(0);
        for (; ok && !w.done(); w.next_item()) {
            const LinRole& R = p.lin.role[w.role];
            const float lg = decay_log2(p.lin.log_decay[w.h]);
            for (; w.k < w.chunks; ++w.k, ++g) {
                if (!(ok = (static_cast<int>(g) + 1 == sm.total || convert(g + 1)) && wait(&sm.o_full[g & 1], g >> 1))) break;
                fence_after();
                const int ea = sm.exps[g % RING][0][i >> 4], nc = w.valid();
                // out = alpha_o 2^ea (g^e 2^eX OI + 2^ef OX), each power in two factors that stay inside fp32's range
                const int ei = ea + sm.state_exp[g % RING], ex = ea + sm.norm[g % RING][i >> 4] + R.alpha_u_exp + 20;
                const float fi = pow2i(ei / 2), fx = pow2i(ex / 2);
                const float gi = R.alpha_o * pow2i(ei - ei / 2) *
                                 exp2f(lg * static_cast<float>(w.rev ? max(0, nc - 1 - i) : i + 1));
                const float gx = R.alpha_o * pow2i(ex - ex / 2);
                const int t = w.token() + i;
                float* row = static_cast<float*>(R.out) + (static_cast<long long>(w.b) * p.lin.T + t) * R.ldo + w.h * D;
#pragma unroll 1
                for (int part = 0; part < 8; ++part) {
                    uint32_t oi[8], ox[8];
                    tmem_rows(tmem + quad + kOI + 64 * (g & 1) + 8 * part, oi);
                    tmem_rows(tmem + quad + kOX + 8 * part, ox);
                    tmem_wait(oi);
                    tmem_wait(ox);
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        const float2 v = fma2(mul2(as_float2(oi[2 * k], oi[2 * k + 1]), both(fi)), both(gi),
                                              mul2(mul2(as_float2(ox[2 * k], ox[2 * k + 1]), both(fx)), both(gx)));
                        oi[2 * k] = i < nc ? __float_as_uint(v.x) : 0u;   // not 0 times what is not finite
                        oi[2 * k + 1] = i < nc ? __float_as_uint(v.y) : 0u;
                    }
                    if (t < p.lin.T) {
#pragma unroll
                        for (int k = 0; k < 2; ++k)
                            *reinterpret_cast<uint4*>(row + 8 * part + 4 * k) =
                                make_uint4(oi[4 * k], oi[4 * k + 1], oi[4 * k + 2], oi[4 * k + 3]);
                    }
                }
                fence_before();
                arrive(&sm.o_free[g & 1]);
            }
            // tokens past the last chunk
            float* po = static_cast<float*>(R.out) + static_cast<long long>(w.b) * p.lin.T * R.ldo + w.h * D;
            const long long z0 = static_cast<long long>(w.chunks) * C, pieces = (p.lin.T - z0) * (D / 4);
            for (long long q = threadIdx.x - 32 * kOutWarp; q < pieces; q += 128)
                *reinterpret_cast<uint4*>(po + (z0 + q / (D / 4)) * R.ldo + q % (D / 4) * 4) = make_uint4(0, 0, 0, 0);
        }
    } else {
        // ---- a and b into pairs
        const int own = warp - kConvertWarp;
        bool ok = true;
        Walk<Tc32Params> w(p);
        for (; ok && w.skip_empty(); ++w.k, ++g) {
            const int s = g % STAGES, nc = w.valid();
            if (!(ok = wait(&sm.full[s], g / STAGES))) break;
#pragma unroll 1
            for (int unit = 0; unit < 4; ++unit) {
                const int tensor = unit < 2 ? 1 : 0, group = 2 * own + (unit & 1);
                convert_tokens(sm.stage[s][tensor][0], group, nc, &sm.exps[g % RING][tensor][group]);
            }
            fence_proxy_async_smem();
            arrive(&sm.ready_ab[s]);
        }
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

int linattn_tc32_launch(int roles, const LinParams& lin, cudaStream_t st)
{
    Tc32Params p{};
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
        if ((rc = token_map(&p.map[i].a, r.a, r.lda, lin, C, true)) != SRWM_OK ||
            (rc = token_map(&p.map[i].b, r.b, r.ldb, lin, C, true)) != SRWM_OK ||
            (rc = token_map(&p.map[i].c, r.c, r.ldc, lin, C, true)) != SRWM_OK)
            return rc;
    }
    static std::atomic<int> sms[kMaxDevices];   // 0: not asked yet
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= kMaxDevices) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    constexpr int smem = static_cast<int>(sizeof(Smem32));
    static_assert(smem <= 227 * 1024, "shared memory of one CTA");
    int n_sm = sms[dev].load();
    if (n_sm == 0) {
        if (cudaDeviceGetAttribute(&n_sm, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess ||
            cudaFuncSetAttribute(reinterpret_cast<const void*>(linattn_tc32_kernel),
                                 cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) {
            cudaGetLastError();
            return SRWM_ERR_CUDA;
        }
        sms[dev].store(n_sm);
    }
    linattn_tc32_kernel<<<p.items < n_sm ? p.items : n_sm, kThreads, smem, st>>>(p);
    return launched();
}

}  // namespace srwm
