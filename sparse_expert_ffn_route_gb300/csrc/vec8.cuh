// vec8.cuh -- eight consecutive values of a row in fp32, bf16 or fp16: loads, stores and what they are in fp32.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "device_util.cuh"
#include "moe.h"

namespace moe {

__device__ __forceinline__ float to_f32(float v) { return v; }
__device__ __forceinline__ float to_f32(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f32(__half v) { return __half2float(v); }
__device__ __forceinline__ void from_f32(float &d, float v) { d = v; }
__device__ __forceinline__ void from_f32(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void from_f32(__half &d, float v) { d = __float2half_rn(v); }

__device__ __forceinline__ void pair_to_f32(const float *p, float &a, float &b)
{
    a = p[0];
    b = p[1];
}
__device__ __forceinline__ void pair_to_f32(const __nv_bfloat16 *p, float &a, float &b)
{
    const uint32_t w = *reinterpret_cast<const uint32_t *>(p);
    a = __uint_as_float(w << 16);
    b = __uint_as_float(w & 0xffff0000u);
}
__device__ __forceinline__ void pair_to_f32(const __half *p, float &a, float &b)
{
    const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(p));
    a = f.x;
    b = f.y;
}
__device__ __forceinline__ void pair_from_f32(float *p, float a, float b)
{
    p[0] = a;
    p[1] = b;
}
__device__ __forceinline__ void pair_from_f32(__nv_bfloat16 *p, float a, float b)
{
    *reinterpret_cast<__nv_bfloat162 *>(p) = __floats2bfloat162_rn(a, b);
}
__device__ __forceinline__ void pair_from_f32(__half *p, float a, float b)
{
    *reinterpret_cast<__half2 *>(p) = __floats2half2_rn(a, b);
}

// as they lie in memory: 16 bytes, or 32 of fp32
template <typename T>
struct Vec8 {
    static constexpr int kWords = sizeof(T) / 2;   // 16-byte words
    union __align__(16) {
        uint4 w[kWords];
        T t[8];
    };
    __device__ Vec8() {}
    __device__ __forceinline__ void load(const T *p)
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = reinterpret_cast<const uint4 *>(p)[i];
    }
    __device__ __forceinline__ void store(T *p) const
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) reinterpret_cast<uint4 *>(p)[i] = w[i];
    }
    __device__ __forceinline__ void zero()
    {
#pragma unroll
        for (int i = 0; i < kWords; ++i) w[i] = make_uint4(0, 0, 0, 0);
    }
    __device__ __forceinline__ void fill(float v)
    {
#pragma unroll
        for (int i = 0; i < 8; ++i) from_f32(t[i], v);
    }
    // all eight in fp32, two at a time: one instruction a value, and one for two of them back
    __device__ __forceinline__ void get(float (&f)[8]) const
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) pair_to_f32(t + 2 * i, f[2 * i], f[2 * i + 1]);
    }
    __device__ __forceinline__ void set(const float (&f)[8])
    {
#pragma unroll
        for (int i = 0; i < 4; ++i) pair_from_f32(t + 2 * i, f[2 * i], f[2 * i + 1]);
    }
};

// f(T()) with the C++ type of a MOE_DTYPE_* code
template <typename F>
auto with_dtype(int dtype, F &&f)
{
    switch (dtype) {
    case MOE_DTYPE_BF16: return f(__nv_bfloat16());
    case MOE_DTYPE_F16: return f(__half());
    default: return f(float());
    }
}

}  // namespace moe
