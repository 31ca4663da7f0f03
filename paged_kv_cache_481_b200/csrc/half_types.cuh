// The two 16-bit storage types (fp16, bf16) behind one set of names, and the
// 8-bit code types of the block-scaled cache.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include <cstdint>

namespace pa {

template <bool kBf16>
struct Half16;

template <>
struct Half16<false> {
    using T2 = __half2;
    // two values of a packed pair, and back (round to nearest even)
    static __device__ __forceinline__ float2 unpack(uint32_t v)
    {
        return __half22float2(*reinterpret_cast<const __half2 *>(&v));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __half2 h = __floats2half2_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

template <>
struct Half16<true> {
    using T2 = __nv_bfloat162;
    static __device__ __forceinline__ float2 unpack(uint32_t v)
    {
        return make_float2(__uint_as_float(v << 16), __uint_as_float(v & 0xffff0000u));
    }
    static __device__ __forceinline__ uint32_t pack(float lo, float hi)
    {
        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&h);
    }
};

// Largest magnitudes of the even and the odd elements of 16 values.
template <typename T2>
__device__ __forceinline__ uint32_t abs_max_pairs(const uint4 &a, const uint4 &b)
{
    const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    T2 m = __habs2(*reinterpret_cast<const T2 *>(&w[0]));
#pragma unroll
    for (int i = 1; i < 8; ++i)
        m = __hmax2(m, __habs2(*reinterpret_cast<const T2 *>(&w[i])));
    return *reinterpret_cast<const uint32_t *>(&m);
}

// Largest code magnitude.
template <bool kE4m3>
__device__ __forceinline__ constexpr float code_top()
{
    return kE4m3 ? 448.0f : 127.0f;
}

// Four values already divided by their scale (at most the top in magnitude) as
// four codes.  Added to 1.5 * 2^23, a small number is rounded to an integer,
// half to even, that stands in the low bits of the sum.
template <bool kE4m3>
__device__ __forceinline__ uint32_t encode4(float a, float b, float c, float d)
{
    if constexpr (kE4m3) {
        const uint32_t lo = __nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3);
        const uint32_t hi = __nv_cvt_float2_to_fp8x2(make_float2(c, d), __NV_SATFINITE, __NV_E4M3);
        return lo | (hi << 16);
    } else {
        const float k = 12582912.0f;
        const uint32_t lo = __byte_perm(__float_as_uint(__fadd_rn(a, k)), __float_as_uint(__fadd_rn(b, k)), 0x0040);
        const uint32_t hi = __byte_perm(__float_as_uint(__fadd_rn(c, k)), __float_as_uint(__fadd_rn(d, k)), 0x0040);
        return __byte_perm(lo, hi, 0x5410);
    }
}

// Two codes (low 16 bits) as the numbers they are.
template <bool kE4m3>
__device__ __forceinline__ float2 decode2(uint32_t c)
{
    if constexpr (kE4m3) {
        const __half2_raw h = __nv_cvt_fp8x2_to_halfraw2(__nv_fp8x2_storage_t(c & 0xffffu), __NV_E4M3);
        return __half22float2(__half2(h));
    } else {
        return make_float2(float(int8_t(c & 0xffu)), float(int8_t((c >> 8) & 0xffu)));
    }
}

} // namespace pa
