// srwm_linattn_tc.cuh -- what the tcgen05 kernels of the linear attention share:
// PTX wrappers, the walk over items and chunks, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include <cstdint>
#include <mutex>

#include "srwm.h"
#include "srwm_f2.cuh"
#include "srwm_linattn.cuh"
#include "srwm_linattn_tc.h"

namespace srwm {
namespace tc {

constexpr int D = 64, C = 128;   // width, tokens of a chunk
constexpr int kMaxDevices = 64;

// Shared-memory matrix descriptor of a 128-byte swizzled tile: atoms of eight
// 128-byte rows, 1024 bytes apart.  K-major operands (rows = M or N, columns =
// K) step 32 bytes per 16 of K inside the rows; MN-major ones (rows = K,
// columns = 64 of M or N) step two atoms.  Bits as in the feed-forward products'
// descriptor: address >> 4, both byte offsets >> 4, version 1, swizzle mode 2.
__device__ __forceinline__ uint64_t desc128(uint32_t saddr)
{
    return static_cast<uint64_t>((saddr & 0x3FFFFu) >> 4) | (static_cast<uint64_t>(64) << 16) |
           (static_cast<uint64_t>(64) << 32) | (static_cast<uint64_t>(1) << 46) | (static_cast<uint64_t>(2) << 61);
}

// kind::f16, fp32 accumulator, A and B of one type (bf16 or fp16); bits 15, 16: A, B MN-major.
__host__ __device__ constexpr uint32_t idesc(bool bf16, int M, int N, bool a_mn, bool b_mn)
{
    return (1u << 4) | (bf16 ? (1u << 7) | (1u << 10) : 0u) | (a_mn ? 1u << 15 : 0u) | (b_mn ? 1u << 16 : 0u) |
           (static_cast<uint32_t>(N >> 3) << 17) | (static_cast<uint32_t>(M >> 4) << 24);
}

template <bool ACC>
__device__ __forceinline__ void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t id)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(id), "n"(ACC ? 1 : 0)
        : "memory");
}
template <bool ACC>
__device__ __forceinline__ void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t id)
{
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d),
        "r"(a), "l"(b), "r"(id), "n"(ACC ? 1 : 0)
        : "memory");
}
// One lane of a converged warp.
__device__ __forceinline__ bool elect()
{
    uint32_t yes;
    asm volatile(
        "{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(yes));
    return yes != 0;
}
// Arrives on `bar` once every product issued before has completed.
__device__ __forceinline__ void commit(uint64_t* bar)
{
    asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_u32(bar))
                 : "memory");
}
__device__ __forceinline__ void fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive(uint64_t* bar)
{
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Tensor memory loads return before their registers are written; tmem_wait
// names the registers, so that no use of them moves ahead of it.
#define SRWM_R16(c, r)                                                                                                 \
    c(r[0]), c(r[1]), c(r[2]), c(r[3]), c(r[4]), c(r[5]), c(r[6]), c(r[7]), c(r[8]), c(r[9]), c(r[10]), c(r[11]),       \
        c(r[12]), c(r[13]), c(r[14]), c(r[15])
#define SRWM_R8(c, r) c(r[0]), c(r[1]), c(r[2]), c(r[3]), c(r[4]), c(r[5]), c(r[6]), c(r[7])
#define SRWM_L8 "{%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
#define SRWM_L16 "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"

// 8 or 16 columns of the warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tmem_rows(uint32_t addr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 " SRWM_L8 : SRWM_R8("=r", r) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_rows(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x16.b32 " SRWM_L16 : SRWM_R16("=r", r) : "r"(addr) : "memory");
}
// 16 or 32 columns of the warp's first 16 lanes, as two or four 16 x 8 accumulator
// fragments: thread l holds (l / 4, 2 (l % 4)), the next column, and both eight lanes below.
__device__ __forceinline__ void tmem_frag16(uint32_t addr, uint32_t (&r)[8])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 " SRWM_L8 : SRWM_R8("=r", r) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_frag32(uint32_t addr, uint32_t (&r)[16])
{
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x4.b32 " SRWM_L16 : SRWM_R16("=r", r) : "r"(addr) : "memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[8])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : SRWM_R8("+r", r)::"memory");
}
__device__ __forceinline__ void tmem_wait(uint32_t (&r)[16])
{
    asm volatile("tcgen05.wait::ld.sync.aligned;" : SRWM_R16("+r", r)::"memory");
}
// 8 columns of the warp's 32 lanes, one lane per thread.
__device__ __forceinline__ void tmem_store8(uint32_t addr, const uint32_t (&r)[8])
{
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"r"(addr), "r"(r[0]),
                 "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
__device__ __forceinline__ void tmem_store_wait() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

__device__ __forceinline__ uint32_t pack_bf16(float x, float y)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack_bf16(float2 v) { return pack_bf16(v.x, v.y); }
__device__ __forceinline__ float2 unpack_bf16(uint32_t v)
{
    return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
}
// Takes the bf16 of both out of v.
__device__ __forceinline__ uint32_t take_bf16(float2& v)
{
    const uint32_t h = pack_bf16(v);
    v = fma2(unpack_bf16(h), both(-1.f), v);
    return h;
}
__device__ __forceinline__ float2 as_float2(uint32_t x, uint32_t y) { return make_float2(__uint_as_float(x), __uint_as_float(y)); }

__device__ __forceinline__ void lds128(uint32_t addr, uint32_t (&v)[4])
{
    asm volatile("ld.shared.v4.u32 {%0,%1,%2,%3}, [%4];" : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]) : "r"(addr));
}
__device__ __forceinline__ void sts128(uint32_t addr, const uint32_t (&v)[4])
{
    asm volatile("st.shared.v4.u32 [%0], {%1,%2,%3,%4};" ::"r"(addr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]) : "memory");
}

// The CTA's items (a stream in a role) and their chunks, as every warp walks them.
template <class Params>
struct Walk {
    const Params& p;
    int item, role, b, h, n, chunks, k;
    bool rev;
    __device__ explicit Walk(const Params& params) : p(params), item(static_cast<int>(blockIdx.x)) { open(); }
    __device__ bool done() const { return item >= p.items; }
    __device__ void open()
    {
        k = 0;
        chunks = 0;
        if (done()) return;
        role = item % p.roles;
        const int stream = item / p.roles;
        b = stream / p.lin.H;
        h = stream % p.lin.H;
        n = p.lin.lengths ? min(max(p.lin.lengths[b], 0), p.lin.T) : p.lin.T;
        rev = p.lin.role[role].reverse != 0;
        chunks = (n + C - 1) / C;
    }
    __device__ void next_item()
    {
        item += static_cast<int>(gridDim.x);
        open();
    }
    // The next chunk, over the ends of items; false at the end of the list.
    __device__ bool skip_empty()
    {
        while (!done() && k >= chunks) next_item();
        return !done();
    }
    __device__ int token() const { return (rev ? chunks - 1 - k : k) * C; }
    __device__ int valid() const { return min(C, n - token()); }
    // Rows that TMA fills with other tokens' values although they are not valid.
    __device__ bool dirty() const { return valid() < C && n < p.lin.T; }
};

// Waits for phase `parity` of `bar`; false, with the CTA marked to end, when it does not come.
static __device__ __forceinline__ bool wait_bounded(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort,
                                                    unsigned* status)
{
    if (mbar_wait_bounded(bar, parity, limit_ns) && !*abort) return true;
    *abort = 1;
    atomicOr(status, kStatusTimeout);
    return false;
}

// The part of a warp's wait that spins, out of line: six kinds of warps share an
// instruction cache, and their loops have to stay in it.  All of its lanes get one
// answer: a phase that ends just at the limit must not part them, since the
// products and the tensor memory accesses that follow take whole warps.
static __device__ __noinline__ bool wait_slow(uint64_t* bar, uint32_t parity, uint64_t limit_ns, volatile int* abort, unsigned* status)
{
    return __all_sync(0xffffffffu, wait_bounded(bar, parity, limit_ns, abort, status));
}

// What a CTA's last copies may take, whatever limit its other waits have.
constexpr uint64_t kDrainLimitNs = 1000000000ull;

// The loader's end, after `chunks` loads into the stages in turn: the shared memory may only be given up once those
// that may still be in flight have landed, whose order is not given.
template <int N>
__device__ __forceinline__ void drain_loads(uint64_t (&full)[N], uint32_t chunks)
{
    for (uint32_t c = chunks > N ? chunks - N : 0; c < chunks; ++c) mbar_wait_bounded(&full[c % N], (c / N) & 1u, kDrainLimitNs);
}

// Tensor memory and the operands' shared memory may only be given up once the products issued have completed.  After a
// timeout, of whichever warp, nobody has waited for the last of them: some microseconds' work, given a millisecond.
static __device__ __noinline__ void let_products_end()
{
    const uint64_t t0 = globaltimer_ns();
    while (globaltimer_ns() - t0 < 1000000ull) {
    }
    __syncwarp();
}

inline PFN_cuTensorMapEncodeTiled_v12000 encoder()
{
    static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
    static std::once_flag once;
    std::call_once(once, [] {
        void* q = nullptr;
        cudaDriverEntryPointQueryResult r;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) == cudaSuccess &&
            r == cudaDriverEntryPointSuccess)
            fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(q);
        else
            cudaGetLastError();
    });
    return fn;
}

// {d, H, T, B} of token rows ld elements apart, boxes of `rows` tokens by 128 bytes of one stream.
inline int token_map(CUtensorMap* map, const void* base, long long ld, const LinParams& p, int rows, bool fp32)
{
    auto enc = encoder();
    if (!enc) return SRWM_ERR_CUDA;
    const cuuint64_t dims[4] = {D, static_cast<cuuint64_t>(p.H), static_cast<cuuint64_t>(p.T), static_cast<cuuint64_t>(p.B)};
    const cuuint64_t e = fp32 ? 4 : 2;
    const cuuint64_t strides[3] = {e * D, static_cast<cuuint64_t>(ld) * e, static_cast<cuuint64_t>(ld) * e * p.T};
    const cuuint32_t box[4] = {static_cast<cuuint32_t>(128 / e), 1, static_cast<cuuint32_t>(rows), 1}, one[4] = {1, 1, 1, 1};
    const CUresult r = enc(map, fp32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4,
                           const_cast<void*>(base), dims, strides, box, one, CU_TENSOR_MAP_INTERLEAVE_NONE,
                           CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_128B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? SRWM_OK : SRWM_ERR_CUDA;
}

}  // namespace tc
}  // namespace srwm
