// gated_kept.cuh -- what the gated block's forward pass keeps of an element for the backward one:
// the two factors that multiply dh,
//   A = u s (1 + g (1 - s)) = dh/dg  and  B = g s = dh/du,  s = sigmoid(g),
// in 16 bits each, A in the word of `g` and B in that of `u`, each with an exponent of its own: A
// grows with u and B with g, dw_gate is made of the one and dw_up of the other, so neither may lose
// bits to the other's size.
//
// fp16: the fp16 numbers themselves.  Off by at most half an fp16 step, infinite from 65520 up.
//
// bf16: a sign and 15 bits that number the magnitudes in order, with steps of
//   2^-10 of the value (10 bits of mantissa)  from 2^-12 to 2^4,
//   2^-7 (bf16's own)                          from 2^-84 to 2^-12 and from 2^4 to 2^60,
// smaller ones to within 2^-92; NaN for NaN, infinity and what is larger.  An eighth of bf16's error
// where the factors of ordinary layers lie and never more than it, at the price of the exponents at the
// far ends.
//
// Gradients' error against 64 bits (norms; an fp32 pass rounded once has 1.66e-3 and 2.1e-4): bf16
// 2.4e-3 with both factors of ordinary size and 2.9e-3 outside, fp16 3.6e-4, whatever the ratio of g to
// u.  The rest is the rounding of dg and du, the tensor cores' operands.  (g and u rounded to the type
// instead: 2.9 to 3.1e-3 and 3.6 to 3.9e-4.  Both factors as whole numbers under one exponent, the
// larger's: 2.4e-3 and 3.1e-4 where g and u are of one size, but the smaller factor is noise where they
// are not, 0.2 at a ratio of 1000.  fp32 would double what both passes move.)
#pragma once

#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <stdint.h>

namespace moe {

template <bool FP16>
struct Kept;

template <>
struct Kept<true> {
    static __device__ __forceinline__ uint32_t code(float v) { return __half_as_ushort(__float2half_rn(v)); }
    // of a code in the upper half of a word
    static __device__ __forceinline__ float value(uint32_t w) { return __half2float(__ushort_as_half((unsigned short)(w >> 16))); }
};

// Over each range of one step the code of a magnitude is its fp32 bits without those below the step
// (rounded, halves up) plus a constant: with m the bits' part inside the fine range, m >> 13 and what is
// left of them >> 16.  2^-84 is added first and taken off last, so that zero has code 0 and what is
// smaller than 2^-84 needs no case of its own.
template <>
struct Kept<false> {
    static constexpr int FROM = (127 - 84) << 23, FINE = (127 - 12) << 23, COARSE = (127 + 4) << 23;   // fp32 bits
    static constexpr int FINE_CODE = (FINE - FROM) >> 16;
    static constexpr int NAN_CODE = 0x7fff;

    static __device__ __forceinline__ uint32_t code(float v)
    {
        const int b = __float_as_int(fabsf(v) + __int_as_float(FROM));
        const int m = min(max(b - FINE, 0), COARSE - FINE);
        const int c = min(((m + (1 << 12) + (FINE_CODE << 13)) >> 13) + ((b - m + (1 << 15) - FINE) >> 16), NAN_CODE);
        return (uint32_t)c | (__float_as_uint(v) >> 16 & 0x8000u);
    }

    // of a code in the upper half of a word
    static __device__ __forceinline__ float value(uint32_t w)
    {
        const int c = (int)(w & 0x7fff0000u);
        const int m = min(max(c - (FINE_CODE << 16), 0), (COARSE - FINE) << 3);
        const float v = __int_as_float(c - m + (m >> 3) + (FINE - (FINE_CODE << 16))) - __int_as_float(FROM);
        return __uint_as_float((c == NAN_CODE << 16 ? 0x7fc00000u : __float_as_uint(v)) | (w & 0x80000000u));
    }
};

// h and the two factors of one element
__device__ __forceinline__ float gated(float g, float u, float &A, float &B)
{
    const float s = __fdividef(1.0f, 1.0f + __expf(-g));
    B = g * s;
    A = u * (s + B * (1.0f - s));
    return B * u;
}

}  // namespace moe
