// srwm_check.h -- host-side argument checks shared by the operator entry
// points (linear attention, group norm).
#pragma once

#include <cuda_runtime.h>

#include <cstddef>
#include <cstdint>
#include <initializer_list>

#include "srwm.h"

namespace srwm {

// Bytes of one element of an enum srwm_dtype, 0 for an unknown one.
inline size_t dtype_bytes(int dtype) { return dtype == SRWM_F32 ? 4 : (dtype == SRWM_BF16 || dtype == SRWM_F16) ? 2 : 0; }

inline size_t round256(size_t n) { return (n + 255) / 256 * 256; }

// A range of `rows` rows of `width` bytes, `pitch` bytes apart (pitch >= width);
// a contiguous array is one row.
struct Region {
    const void* p;
    size_t width, pitch;
    long long rows;
};

inline Region flat(const void* p, size_t bytes) { return {p, bytes, bytes, 1}; }

inline size_t span(const Region& r) { return r.rows <= 0 ? 0 : static_cast<size_t>(r.rows - 1) * r.pitch + r.width; }

// Whether two regions share a byte.  Two regions of one pitch may interleave
// (the slices of one packed projection): then they are apart when their rows'
// offsets within the pitch are.
inline bool overlap(const Region& a, const Region& b)
{
    if (!a.p || !b.p || span(a) == 0 || span(b) == 0) return false;
    const uintptr_t a0 = reinterpret_cast<uintptr_t>(a.p), b0 = reinterpret_cast<uintptr_t>(b.p);
    if (!(a0 < b0 + span(b) && b0 < a0 + span(a))) return false;
    if (a.pitch == b.pitch && a.rows > 1 && b.rows > 1) {
        const size_t off = a0 <= b0 ? (b0 - a0) % a.pitch : (a.pitch - (a0 - b0) % a.pitch) % a.pitch;
        return off < a.width || off + b.width > a.pitch;
    }
    return true;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

// Device memory of the current device, or managed memory?
inline int check_device_memory(std::initializer_list<const void*> ptrs)
{
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) {
        cudaGetLastError();
        return SRWM_ERR_CUDA;
    }
    for (const void* p : ptrs) {
        if (!p) continue;
        cudaPointerAttributes attr;
        if (cudaPointerGetAttributes(&attr, p) != cudaSuccess) {
            cudaGetLastError();
            return SRWM_ERR_NOT_DEVICE;
        }
        if (attr.type == cudaMemoryTypeManaged) continue;
        if (attr.type != cudaMemoryTypeDevice || attr.device != dev) return SRWM_ERR_NOT_DEVICE;
    }
    return SRWM_OK;
}

// Launches a kernel that calls griddep_wait() (srwm_mma.cuh) behind one that calls griddep_launch(): its CTAs may be
// placed while the last of the other's still run, instead of some 2 us after them.
template <typename... P, typename... A>
int launch_behind(void (*kernel)(P...), dim3 grid, int threads, int smem, cudaStream_t st, const A&... args)
{
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(static_cast<unsigned>(threads));
    cfg.dynamicSmemBytes = static_cast<size_t>(smem);
    cfg.stream = st;
    cudaLaunchAttribute attr{};
    attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr.val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = &attr;
    cfg.numAttrs = 1;
    if (cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess) return SRWM_OK;
    cudaGetLastError();
    return SRWM_ERR_CUDA;
}

inline int launched() { return cudaGetLastError() == cudaSuccess ? SRWM_OK : SRWM_ERR_CUDA; }

}  // namespace srwm
