// eight.cuh -- eight consecutive elements of a plain matrix in registers: as they lie in
// memory, and as 32-bit values.
#pragma once

#include <cstdint>

#include "mx4.cuh"

namespace ddg {
namespace {

template <typename T> struct Eight { uint32_t w[sizeof(T) * 2]; };

// From a 16-byte aligned address on.
template <typename T>
__device__ __forceinline__ void load8(const T* p, Eight<T>& x) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T) * 2; i += 4) {
        const uint4 v = reinterpret_cast<const uint4*>(p)[i / 4];
        x.w[i] = v.x, x.w[i + 1] = v.y, x.w[i + 2] = v.z, x.w[i + 3] = v.w;
    }
}
__device__ __forceinline__ void unpack8(const Eight<float>& x, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) y[i] = __uint_as_float(x.w[i]);
}
__device__ __forceinline__ void unpack8(const Eight<__nv_bfloat16>& x, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        y[2 * i] = __uint_as_float(x.w[i] << 16);
        y[2 * i + 1] = __uint_as_float(x.w[i] & 0xffff0000u);
    }
}
__device__ __forceinline__ void unpack8(const Eight<__half>& x, float (&y)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const float2 v = __half22float2(*reinterpret_cast<const __half2*>(&x.w[i]));
        y[2 * i] = v.x;
        y[2 * i + 1] = v.y;
    }
}
// Two values to nearest in one instruction.
template <typename T> __device__ __forceinline__ uint32_t pair_of(float a, float b);
template <> __device__ __forceinline__ uint32_t pair_of<__nv_bfloat16>(float a, float b) {
    uint32_t w;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
template <> __device__ __forceinline__ uint32_t pair_of<__half>(float a, float b) {
    uint32_t w;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(b), "f"(a));
    return w;
}
template <typename T>
__device__ __forceinline__ void pack8(T* p, const float (&y)[8]) {
    if constexpr (sizeof(T) == 4) {
        reinterpret_cast<float4*>(p)[0] = make_float4(y[0], y[1], y[2], y[3]);
        reinterpret_cast<float4*>(p)[1] = make_float4(y[4], y[5], y[6], y[7]);
    } else {
        *reinterpret_cast<uint4*>(p) = make_uint4(pair_of<T>(y[0], y[1]), pair_of<T>(y[2], y[3]), pair_of<T>(y[4], y[5]), pair_of<T>(y[6], y[7]));
    }
}

}  // namespace
}  // namespace ddg
