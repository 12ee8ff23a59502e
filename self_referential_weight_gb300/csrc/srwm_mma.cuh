// srwm_mma.cuh -- warp-level fp16 matrix products with fp32 accumulation
// (mma.sync m16n8k16), the loads of their fragments, 16-byte asynchronous
// copies, and the order of a call's kernels, as inline PTX.
#pragma once

#include <cuda_fp16.h>

#include <cstdint>

#include "srwm_f2.cuh"

namespace srwm {

// c[16x8] += a[16x16] b[16x8].  Lane l holds, with r = l / 4 and x = 2 (l % 4):
// c = (r, x), (r, x + 1), (r + 8, x), (r + 8, x + 1); a = pairs of columns at
// (r, x), (r + 8, x), (r, x + 8), (r + 8, x + 8); b = pairs of rows at (x, r), (x + 8, r).
__device__ __forceinline__ void mma16816(float (&c)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

// Four 8x8 blocks of 16-bit values; lanes 8i .. 8i + 7 give the row addresses of block i.
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

__device__ __forceinline__ void ldmatrix4_trans(uint32_t (&r)[4], uint32_t addr)
{
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// 16 bytes global -> shared; zeros instead of reading when !valid.
__device__ __forceinline__ void cp_async16(uint32_t dst, const void* src, bool valid)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(valid ? 16 : 0) : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint32_t pack_half2(float x, float y)
{
    const __half2 h = __floats2half2_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&h);
}

__device__ __forceinline__ float2 unpack_half2(uint32_t v)
{
    return __half22float2(*reinterpret_cast<const __half2*>(&v));
}

// (x, y) as a high and a low pair of fp16: 22 bits of each.
__device__ __forceinline__ void split_half2(float x, float y, uint32_t& hi, uint32_t& lo)
{
    hi = pack_half2(x, y);
    const float2 h = unpack_half2(hi);
    lo = pack_half2(x - h.x, y - h.y);
}

// The same with two fp32 operations per instruction.
__device__ __forceinline__ void split_half2_2(float2 v, uint32_t& hi, uint32_t& lo)
{
    hi = pack_half2(v.x, v.y);
    const float2 rest = fma2(unpack_half2(hi), both(-1.f), v);
    lo = pack_half2(rest.x, rest.y);
}

// For the kernels of one call that follow each other closely (launch_behind in srwm_check.h): a kernel lets the next be
// placed as soon as all of its own CTAs are; the next waits for it to have completed.
__device__ __forceinline__ void griddep_launch() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void griddep_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

}  // namespace srwm
