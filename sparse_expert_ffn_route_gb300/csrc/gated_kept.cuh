// gated_kept.cuh -- what the gated block's forward pass keeps of an element for the backward one:
// both factors that multiply dh,
//   A = u s (1 + g (1 - s)) = dh/dg  and  B = g s = dh/du,  s = sigmoid(g),
// in 32 bits, one word: an exponent e that the two share and two whole numbers a, b with
// A = a 2^e 2/H, B = b 2^e 2/H, |a|, |b| <= H.  bf16: 8 bits of e, H = 2047; fp16: 5 bits, H = 5792
// (two numbers of 2H + 1 values fill 27 bits).  Each is off by at most max(|A|, |B|) / H, an eighth
// of a bf16 number's half step and about half an fp16 one's.
//
// Why: g and u in the 16-bit type, in as many bytes, put the gradients' error at 1.8 times that of an
// fp32 pass rounded once; this puts it at 1.45, the rounding of dg and du as operands of the tensor
// cores being what is left.  (In fp32 they would double what both passes move.)
//
// fp16 holds e from -13 to 16, bf16 from -103: smaller factors keep the step of the least e (4e-8 in
// fp16, less than its own subnormal step).  A factor that is NaN, infinite or from 2^17 (fp16) or 2^127 (bf16) up makes the
// word stand for NaN.
#pragma once

#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

template <bool FP16>
struct Kept {
    static constexpr int H = FP16 ? 5792 : 2047;
    static constexpr uint32_t RADIX = 2 * H + 1;
    static constexpr int SHIFT = FP16 ? 27 : 24;                 // of the exponent's code
    static constexpr int BIAS = FP16 ? 14 : 127;                 // e = code - BIAS
    static constexpr uint32_t BAD = FP16 ? 31u : 255u, TOP = FP16 ? 30u : 253u;   // NaN, the largest e
    static constexpr int LEAST = FP16 ? 1 : 24;                  // the least e: 2^-e H/2 is finite

    static __device__ __forceinline__ uint32_t pack(float A, float B)
    {
        const uint32_t most = max(__float_as_uint(A) & 0x7fffffffu, __float_as_uint(B) & 0x7fffffffu);
        const int code = max((int)(most >> 23) - 127 + BIAS, LEAST);
        if (code > (int)TOP) return BAD << SHIFT;
        const float f = __uint_as_float((uint32_t)(127 + BIAS - code) << 23) * (0.5f * H);   // 2^-e H/2
        const uint32_t a = (uint32_t)(__float2int_rn(A * f) + H), b = (uint32_t)(__float2int_rn(B * f) + H);
        return (uint32_t)code << SHIFT | (a * RADIX + b);
    }

    static __device__ __forceinline__ void unpack(uint32_t w, float &A, float &B)
    {
        const uint32_t code = w >> SHIFT, q = w & ((1u << SHIFT) - 1u), a = q / RADIX, b = q - a * RADIX;
        const float f = code == BAD ? __uint_as_float(0x7fc00000u)
                                    : __uint_as_float((code + 127u - BIAS) << 23) * (2.0f / H);   // 2^e 2/H
        A = (float)((int)a - H) * f;
        B = (float)((int)b - H) * f;
    }
};

// h and the kept word of one element
__device__ __forceinline__ float gated(float g, float u, float &A, float &B)
{
    const float s = __fdividef(1.0f, 1.0f + __expf(-g));
    B = g * s;
    A = u * (s + B * (1.0f - s));
    return B * u;
}

}  // namespace moe
