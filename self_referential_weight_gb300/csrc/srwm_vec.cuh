// srwm_vec.cuh -- 16-byte vectors of an operator's elements as fp32 values, and
// the sigmoid of its activations.
#pragma once

#include <cstddef>

#include "srwm_elem.cuh"
#include "srwm_mma.cuh"
#include "srwm_ptx.cuh"

namespace srwm {

template <typename E>
constexpr int vec = 16 / static_cast<int>(sizeof(E));

__device__ __forceinline__ void unpack(const uint4& u, float (&f)[4], float)
{
    f[0] = __uint_as_float(u.x), f[1] = __uint_as_float(u.y), f[2] = __uint_as_float(u.z), f[3] = __uint_as_float(u.w);
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8], __nv_bfloat16)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        f[2 * k] = __uint_as_float(w[k] << 16);
        f[2 * k + 1] = __uint_as_float(w[k] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack(const uint4& u, float (&f)[8], __half)
{
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
        const float2 v = unpack_half2(w[k]);
        f[2 * k] = v.x;
        f[2 * k + 1] = v.y;
    }
}
__device__ __forceinline__ uint4 pack(const float (&f)[4], float)
{
    return make_uint4(__float_as_uint(f[0]), __float_as_uint(f[1]), __float_as_uint(f[2]), __float_as_uint(f[3]));
}
__device__ __forceinline__ uint32_t pack2(float x, float y, __nv_bfloat16)
{
    const __nv_bfloat162 v = __floats2bfloat162_rn(x, y);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ uint32_t pack2(float x, float y, __half) { return pack_half2(x, y); }
template <typename E>
__device__ __forceinline__ uint4 pack(const float (&f)[8], E)
{
    return make_uint4(pack2(f[0], f[1], E{}), pack2(f[2], f[3], E{}), pack2(f[4], f[5], E{}), pack2(f[6], f[7], E{}));
}

template <typename E>
__device__ __forceinline__ uint4 load_vec(const void* p, size_t element)
{
    return __ldg(reinterpret_cast<const uint4*>(static_cast<const E*>(p) + element));
}
template <typename E>
__device__ __forceinline__ void store_vec(void* p, size_t element, const uint4& v)
{
    *reinterpret_cast<uint4*>(static_cast<E*>(p) + element) = v;
}

// Four neighbouring elements: half a vector of the 16-bit types.
template <typename E> struct Quad { using type = uint2; };
template <> struct Quad<float> { using type = uint4; };

template <typename E>
__device__ __forceinline__ typename Quad<E>::type load_quad(const void* p, size_t element)
{
    return __ldg(reinterpret_cast<const typename Quad<E>::type*>(static_cast<const E*>(p) + element));
}
__device__ __forceinline__ void unpack_quad(const uint4& u, float (&f)[4], float) { unpack(u, f, 0.f); }
template <typename E>
__device__ __forceinline__ void unpack_quad(const uint2& u, float (&f)[4], E)
{
    float e[8];
    unpack(make_uint4(u.x, u.y, 0u, 0u), e, E{});
    f[0] = e[0], f[1] = e[1], f[2] = e[2], f[3] = e[3];
}
__device__ __forceinline__ uint4 pack_quad(const float (&f)[4], float) { return pack(f, 0.f); }
template <typename E>
__device__ __forceinline__ uint2 pack_quad(const float (&f)[4], E) { return make_uint2(pack2(f[0], f[1], E{}), pack2(f[2], f[3], E{})); }
template <typename E>
__device__ __forceinline__ void store_quad(void* p, size_t element, const typename Quad<E>::type& v)
{
    *reinterpret_cast<typename Quad<E>::type*>(static_cast<E*>(p) + element) = v;
}

// sigmoid(z), good to about (|z| + 3) 2^-23 of itself for z < 0, where the rounding of exp's argument grows with it,
// and to 3 * 2^-23 above: exp underflows to 0 and overflows to infinity, whose reciprocal is 0.
__device__ __forceinline__ float sigmoid(float z)
{
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(-1.4426950408889634f * z));
    return rcp_approx(1.f + e);
}

}  // namespace srwm
