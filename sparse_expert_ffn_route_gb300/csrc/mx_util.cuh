// mx_util.cuh -- the MXFP4 rules shared by the quantiser and the products' epilogue.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

// Scale byte and the factor 2^-e of a block whose largest magnitude is `amax` (as fp32 bits):
// e = floor(log2 amax) - 2, held as e + 127 and no less than 0; byte 255 and factor 0 for a NaN or
// an infinity (whose bits are the largest of the block's).
__device__ __forceinline__ uint32_t mx_scale(uint32_t amax_bits, float &factor)
{
    const uint32_t ex = amax_bits >> 23;
    const uint32_t sb = ex == 255u ? 255u : ex > 2u ? ex - 2u : 0u;
    factor = ex == 255u ? 0.0f : __uint_as_float((254u - sb) << 23);
    return sb;
}

// 2^(byte - 127); NaN for 255
__device__ __forceinline__ float mx_scale_value(uint32_t sb)
{
    return __uint_as_float(sb == 0 ? 0x00400000u : sb == 255u ? 0x7fc00000u : sb << 23);
}

// two values -> two e2m1 codes (round half to even, saturating at 6), lo in bits 0-3
__device__ __forceinline__ uint32_t e2m1x2(float lo, float hi)
{
    uint32_t r;
    asm("{\n\t.reg .b8 t;\n\tcvt.rn.satfinite.e2m1x2.f32 t, %2, %1;\n\tcvt.u32.u8 %0, t;\n\t}"
        : "=r"(r)
        : "f"(lo), "f"(hi));
    return r;
}

// the values of the two codes in bits 0-3 and 4-7
__device__ __forceinline__ float2 e2m1x2_values(uint32_t byte)
{
    uint32_t h;
    asm("{\n\t.reg .b8 t;\n\tcvt.u8.u32 t, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, t;\n\t}" : "=r"(h) : "r"(byte));
    return __half22float2(*reinterpret_cast<const __half2 *>(&h));
}

}  // namespace moe
