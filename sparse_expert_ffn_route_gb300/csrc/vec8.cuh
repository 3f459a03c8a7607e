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

// as they lie in memory: 16 bytes, or 32 of fp32
template <typename T>
struct Vec8 {
    static constexpr int kWords = sizeof(T) / 2;   // 16-byte words
    union {
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
    __device__ __forceinline__ float get(int i) const { return to_f32(t[i]); }
    __device__ __forceinline__ void set(int i, float v) { from_f32(t[i], v); }
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
