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
    using T = __half;
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
    using T = __nv_bfloat16;
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

// Largest code magnitude.
template <bool kE4m3>
__device__ __forceinline__ constexpr float code_top()
{
    return kE4m3 ? 448.0f : 127.0f;
}

// Two values already divided by their scale, as two codes in the low 16 bits.
template <bool kE4m3>
__device__ __forceinline__ uint32_t encode2(float a, float b)
{
    if constexpr (kE4m3) {
        return uint32_t(__nv_cvt_float2_to_fp8x2(make_float2(a, b), __NV_SATFINITE, __NV_E4M3));
    } else {
        const int ia = int(fminf(fmaxf(rintf(a), -127.0f), 127.0f));
        const int ib = int(fminf(fmaxf(rintf(b), -127.0f), 127.0f));
        return (uint32_t(ia) & 0xffu) | ((uint32_t(ib) & 0xffu) << 8);
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
