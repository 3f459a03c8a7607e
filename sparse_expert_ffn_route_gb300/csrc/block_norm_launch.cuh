// block_norm_launch.cuh -- the launches of block_norm.cuh's kernels for one type of the stream.
#pragma once

#include "block_norm.cuh"

namespace moe {
namespace norm {

template <typename X>
cudaError_t launch_forward(const NormArgs &p, int dtype, cudaStream_t st)
{
    const int threads = norm_threads(p.H, kVecs);
    return with_dtype(dtype, [&](auto yt) {
        using Y = decltype(yt);
        const int ring = kRowStages * p.H * (int)(sizeof(X) + (p.y ? sizeof(Y) : 0) + (p.kind == kGateFull ? sizeof(Y) : 0));
        const int fit = forward_ctas(threads, ring);
        // (three rows a CTA fill its ring; with fewer the kernel of one row a CTA begins sooner)
        if (fit >= 2 && p.T >= 3 * fit * num_sms())
            return launch_kernel(threads <= 448 ? norm_rows_kernel<X, Y, 448> : norm_rows_kernel<X, Y, 512>, dim3(fit * num_sms()),
                                 dim3(threads), ring, st, 1, p);
        return launch_kernel(norm_forward_kernel<X, Y>, dim3(p.T), dim3(threads), 0, st, 1, p);
    });
}

template <typename X>
cudaError_t launch_backward(NormArgs p, int dtype, int parts, cudaStream_t st)
{
    const int threads = norm_threads(p.H, 1);
    return with_dtype(dtype, [&](auto yt) {
        using Y = decltype(yt);
        const int row = (int)RowBytes(p, sizeof(X), sizeof(Y)).total();
        const int ctas = ctas_per_sm(p.H, heavy_backward(p));
        p.stages = backward_stages(row, parts, ctas);
        const auto go = [&](auto kind, auto post, auto pre) {
            constexpr int KIND = decltype(kind)::value;
            constexpr bool POST = decltype(post)::value, PRE = decltype(pre)::value;
            return launch_kernel(ctas * threads <= 768   ? norm_backward_kernel<X, Y, 768, KIND, POST, PRE>
                                 : ctas * threads <= 896 ? norm_backward_kernel<X, Y, 896, KIND, POST, PRE>
                                                         : norm_backward_kernel<X, Y, 1024, KIND, POST, PRE>,
                                 dim3(parts), dim3(threads), (size_t)p.stages * row, st, 1, p);
        };
        using std::integral_constant;
        constexpr std::true_type yes;
        constexpr std::false_type no;
        const bool gate = p.kind == kGateChannel ? p.want_channel : p.kind == kGateNone || p.dgate;
        if (!(p.dout && p.y && p.dx && p.dy && gate && p.want_pre == (p.dn != nullptr) && p.want_post == (p.post != nullptr)))
            return go(integral_constant<int, -1>(), no, no);
        const auto with = [&](auto kind) {
            return p.post ? p.dn ? go(kind, yes, yes) : go(kind, yes, no) : p.dn ? go(kind, no, yes) : go(kind, no, no);
        };
        switch (p.kind) {
        case kGateChannel: return with(integral_constant<int, kGateChannel>());
        case kGateToken: return with(integral_constant<int, kGateToken>());
        case kGateFull: return with(integral_constant<int, kGateFull>());
        default: return with(integral_constant<int, kGateNone>());
        }
    });
}

}  // namespace norm
}  // namespace moe
