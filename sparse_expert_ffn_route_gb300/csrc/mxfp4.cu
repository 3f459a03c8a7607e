// mxfp4.cu -- rows to MXFP4 and back.
//
// A block of 32 values of a row shares the scale 2^e, e = floor(log2(largest magnitude)) - 2 (so
// the largest lands in [4, 8)), held as the byte e + 127; each value is the e2m1 code (sign, two
// exponent bits, one mantissa bit: 0, .5, 1, 1.5, 2, 3, 4, 6) nearest to x / 2^e, ties to the
// even code, magnitudes above 6 held as 6 (the rule of the OCP Microscaling Formats
// specification 1.0, section 6.3).  e is no less than -127; a block of zeros has scale byte 0 and codes
// 0; a block with a NaN or an infinity has scale byte 255, which stands for NaN, and codes 0.
// Everything but the final rounding to a code is exact: the factor is a power of two.
//
// Bound by memory.  A warp takes 1024 consecutive values of a row, 8 a lane in each of 4 steps:
// one or two 16-byte loads a step, all issued before the first use; the 4 lanes of a block
// meet in two shuffles; a step's codes go out as 128 consecutive bytes.
#include <type_traits>

#include "device_util.cuh"
#include "launch.cuh"
#include "moe_internal.cuh"
#include "mx_util.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kSteps = 4;              // 256 values a warp and step
constexpr int kDeqSteps = 4;           // units a lane writes in the dequantiser
constexpr int kSeg = 256 * kSteps;     // values of a row that a warp takes

template <typename T>
struct Vec8;   // 8 consecutive values as loaded

template <>
struct Vec8<float> {
    uint4 a, b;
    __device__ __forceinline__ void load(const float *p)
    {
        a = ld_stream_v4(p);
        b = ld_stream_v4(p + 4);
    }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        v[0] = __uint_as_float(a.x), v[1] = __uint_as_float(a.y), v[2] = __uint_as_float(a.z), v[3] = __uint_as_float(a.w);
        v[4] = __uint_as_float(b.x), v[5] = __uint_as_float(b.y), v[6] = __uint_as_float(b.z), v[7] = __uint_as_float(b.w);
    }
};

template <>
struct Vec8<__nv_bfloat16> {
    uint4 a;
    __device__ __forceinline__ void load(const __nv_bfloat16 *p) { a = ld_stream_v4(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            v[2 * i] = __uint_as_float(w[i] << 16);
            v[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
        }
    }
};

template <>
struct Vec8<__half> {
    uint4 a;
    __device__ __forceinline__ void load(const __half *p) { a = ld_stream_v4(p); }
    __device__ __forceinline__ void get(float (&v)[8]) const
    {
        const uint32_t w[4] = {a.x, a.y, a.z, a.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&w[i]));
            v[2 * i] = f.x;
            v[2 * i + 1] = f.y;
        }
    }
};

template <typename T, bool GATHER>
__global__ void __launch_bounds__(kThreads)
    quantize_kernel(const T *__restrict__ x, long long ldx, long long segs, int per_row, int K,
                    const int32_t *__restrict__ tok, const int32_t *__restrict__ limit, int nx, uint8_t *__restrict__ codes,
                    uint8_t *__restrict__ scales, int32_t *err)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long seg = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
    if (seg >= segs) return;
    const long long row = seg / per_row;
    const int k0 = (int)(seg - row * per_row) * kSeg + lane * 8;
    long long src = row;
    if (GATHER) {
        if (row >= *limit) return;
        src = tok[row];
        if (src < 0 || src >= nx) {   // a bad index: the row's scales become NaN, and it is recorded
            if (lane == 0) atomicOr(err, kErrBadToken);
            src = -1;
        }
    }
    Vec8<T> in[kSteps];
#pragma unroll
    for (int i = 0; i < kSteps; ++i)
        if (k0 + 256 * i < K && src >= 0) in[i].load(x + src * ldx + k0 + 256 * i);
#pragma unroll
    for (int i = 0; i < kSteps; ++i) {
        const int k = k0 + 256 * i;
        // lanes of a block are in or out together (K is a multiple of 32)
        const bool in_row = k < K;
        float v[8];
        uint32_t top = 0;
        if (in_row && src >= 0) {
            in[i].get(v);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max(top, __float_as_uint(v[j]) & 0x7fffffffu);
        } else {
            top = 0x7f800000u;
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = 0.0f;
        }
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 1));
        top = max(top, __shfl_xor_sync(0xffffffffu, top, 2));
        float f;
        const uint32_t sb = mx_scale(top, f);
        uint32_t w = 0;
#pragma unroll
        for (int j = 0; j < 8; j += 2)
            w |= e2m1x2(f == 0.0f ? 0.0f : v[j] * f, f == 0.0f ? 0.0f : v[j + 1] * f) << (4 * j);
        if (in_row) {
            *reinterpret_cast<uint32_t *>(codes + ((row * K + k) >> 1)) = w;
            if ((lane & 3) == 0) scales[(row * K + k) >> 5] = (uint8_t)sb;
        }
    }
}

// Quantised rows in the order of a list: row r from row tok[r] for r < *limit, one warp a row.
// A bad index: NaN scales and a record, as in the quantiser.
__global__ void __launch_bounds__(kThreads)
    gather_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, long long rows, int K,
                  const int32_t *__restrict__ tok, const int32_t *__restrict__ limit, int nx, uint8_t *__restrict__ to_codes,
                  uint8_t *__restrict__ to_scales, int32_t *err)
{
    pdl_wait();
    pdl_launch_dependents();
    const int lane = threadIdx.x & 31;
    const long long row = ((long long)blockIdx.x * kThreads + threadIdx.x) >> 5;
    if (row >= rows || row >= *limit) return;
    const int src = tok[row];
    const bool bad = src < 0 || src >= nx;
    if (bad && lane == 0) atomicOr(err, kErrBadToken);
    const int chunks = K / 32;   // 16 bytes of codes and a scale byte each
    const uint4 *from = reinterpret_cast<const uint4 *>(codes) + (long long)(bad ? 0 : src) * chunks;
    uint4 *to = reinterpret_cast<uint4 *>(to_codes) + row * chunks;
    for (int i0 = lane; i0 < chunks; i0 += 4 * 32) {
        uint4 v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            v[j] = make_uint4(0, 0, 0, 0);
            if (i0 + 32 * j < chunks && !bad) v[j] = __ldg(from + i0 + 32 * j);
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + 32 * j < chunks) to[i0 + 32 * j] = v[j];
    }
    // K is a multiple of 64: an even number of scale bytes a row
    const uint16_t *sf = reinterpret_cast<const uint16_t *>(scales) + (long long)(bad ? 0 : src) * (chunks / 2);
    uint16_t *st = reinterpret_cast<uint16_t *>(to_scales) + row * (chunks / 2);
    for (int i = lane; i < chunks / 2; i += 32) st[i] = bad ? (uint16_t)0xffff : __ldg(sf + i);
}

// A lane writes 16 consecutive bytes a step, so that a warp's stores are 512 consecutive bytes:
// 4 values in fp32 (8, as two stores 32 bytes apart over the warp, wrote 403 MB at 4.9 TB/s; this
// way at 6.5 TB/s), 8 in 16 bits.
__device__ __forceinline__ void put(float *p, const float (&v)[4])
{
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
}

__device__ __forceinline__ void put(__nv_bfloat16 *p, const float (&v)[8])
{
    __nv_bfloat162 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(o);
}

__device__ __forceinline__ void put(__half *p, const float (&v)[8])
{
    __half2 o[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) o[i] = __floats2half2_rn(v[2 * i], v[2 * i + 1]);
    *reinterpret_cast<uint4 *>(p) = *reinterpret_cast<const uint4 *>(o);
}

template <typename T>
__global__ void __launch_bounds__(kThreads)
    dequantize_kernel(const uint8_t *__restrict__ codes, const uint8_t *__restrict__ scales, long long units,
                      T *__restrict__ y)
{
    constexpr int V = 16 / sizeof(T);   // values of a unit: 16 bytes of y, 2 or 4 bytes of codes
    using Codes = typename std::conditional<V == 4, uint16_t, uint32_t>::type;
    pdl_wait();
    pdl_launch_dependents();
    // unit u: values V u .. of the rows laid end to end (K is a multiple of 32)
    const int lane = threadIdx.x & 31;
    const long long u0 = (((long long)blockIdx.x * kThreads + threadIdx.x) >> 5) * (32 * kDeqSteps) + lane;
    uint32_t w[kDeqSteps], sb[kDeqSteps];
#pragma unroll
    for (int i = 0; i < kDeqSteps; ++i)
        if (u0 + 32 * i < units) {
            w[i] = __ldg(reinterpret_cast<const Codes *>(codes) + u0 + 32 * i);
            sb[i] = __ldg(scales + (u0 + 32 * i) / (32 / V));
        }
#pragma unroll
    for (int i = 0; i < kDeqSteps; ++i) {
        if (u0 + 32 * i >= units) return;
        const float s = mx_scale_value(sb[i]);
        float v[V];
#pragma unroll
        for (int j = 0; j < V / 2; ++j) {
            const float2 p = e2m1x2_values(w[i] >> (8 * j));
            v[2 * j] = p.x * s;
            v[2 * j + 1] = p.y * s;
        }
        put(y + (u0 + 32 * i) * V, v);
    }
}

template <typename T>
cudaError_t quantize(const void *x, long long ldx, long long rows, int K, const int32_t *tok, const int32_t *limit, int nx,
                     uint8_t *codes, uint8_t *scales, int32_t *err, cudaStream_t st)
{
    const int per_row = (K + kSeg - 1) / kSeg;
    const long long segs = rows * per_row;
    const dim3 grid((unsigned)((segs * 32 + kThreads - 1) / kThreads));
    return tok ? launch_kernel(quantize_kernel<T, true>, grid, dim3(kThreads), 0, st, 1, static_cast<const T *>(x), ldx,
                               segs, per_row, K, tok, limit, nx, codes, scales, err)
               : launch_kernel(quantize_kernel<T, false>, grid, dim3(kThreads), 0, st, 1, static_cast<const T *>(x), ldx,
                               segs, per_row, K, tok, limit, nx, codes, scales, err);
}

}  // namespace

cudaError_t launch_quantize_mxfp4(const void *x, int dtype, long long ldx, long long rows, int K, const int32_t *tok,
                                  const int32_t *limit, int T, uint8_t *codes, uint8_t *scales, int32_t *err,
                                  cudaStream_t st)
{
    if (dtype == MOE_DTYPE_F32) return quantize<float>(x, ldx, rows, K, tok, limit, T, codes, scales, err, st);
    if (dtype == MOE_DTYPE_BF16) return quantize<__nv_bfloat16>(x, ldx, rows, K, tok, limit, T, codes, scales, err, st);
    return quantize<__half>(x, ldx, rows, K, tok, limit, T, codes, scales, err, st);
}

cudaError_t launch_gather_mxfp4(const uint8_t *codes, const uint8_t *scales, long long rows, int K, const int32_t *tok,
                                const int32_t *limit, int T, uint8_t *to_codes, uint8_t *to_scales, int32_t *err,
                                cudaStream_t st)
{
    const dim3 grid((unsigned)((rows * 32 + kThreads - 1) / kThreads));
    return launch_kernel(gather_kernel, grid, dim3(kThreads), 0, st, 1, codes, scales, rows, K, tok, limit, T, to_codes,
                         to_scales, err);
}

cudaError_t launch_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, long long rows, int K, void *y,
                                    int dtype, cudaStream_t st)
{
    const long long units = rows * K / (dtype == MOE_DTYPE_F32 ? 4 : 8);
    const dim3 grid((unsigned)((units + kThreads * kDeqSteps - 1) / (kThreads * kDeqSteps)));
    if (dtype == MOE_DTYPE_F32)
        return launch_kernel(dequantize_kernel<float>, grid, dim3(kThreads), 0, st, 1, codes, scales, units, (float *)y);
    if (dtype == MOE_DTYPE_BF16)
        return launch_kernel(dequantize_kernel<__nv_bfloat16>, grid, dim3(kThreads), 0, st, 1, codes, scales, units,
                             (__nv_bfloat16 *)y);
    return launch_kernel(dequantize_kernel<__half>, grid, dim3(kThreads), 0, st, 1, codes, scales, units, (__half *)y);
}

}  // namespace moe
