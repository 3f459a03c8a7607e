// block_norm.cu -- the step between two blocks of the residual stream and its gradients:
//   z = y iy post (iy = 1 / sqrt(mean y^2 + eps); z = y without post),  out = a x + b gate z,
//   n = out io pre (io = 1 / sqrt(mean out^2 + eps)).
// Backward, from dout and dn: with w = dn pre, e = dout + io w and c1 = sum w out,
//   d = e - io^3 c1 / H out  (all of out's gradient),  dx = a d,  dz = b gate d,  dgate = b d z,
//   dy = iy (dz post - iy^2 c2 / H y),  c2 = sum dz post y,  dpost = sum_t dz y iy,  dpre = sum_t dn out io.
// c2, and the gate's gradient where it is one number a token, are sums over d, which needs c1; but
//   sum q d = sum q e - (io^3 c1 / H) sum q out,
// so three sums over the row, taken together, give all of them and a row costs one exchange between the
// warps instead of two.
#include "block_norm.cuh"

namespace moe {

using namespace norm;

namespace {

// Sums of the CTAs' parts, 32 columns a CTA, in a fixed order.
__global__ void __launch_bounds__(1024) norm_parts_kernel(const float *part, int parts, int H, float *dpre, float *dpost, float *dchan)
{
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float s_sum[32][32];
    float *to = blockIdx.y == 0 ? dpre : blockIdx.y == 1 ? dpost : dchan;
    if (!to) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, h = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (h < H)
#pragma unroll 8
        for (int i = w; i < parts; i += 32) sum += part[((size_t)i * 3 + blockIdx.y) * H + h];
    s_sum[w][lane] = sum;
    __syncthreads();
    if (w || h >= H) return;
    for (int i = 1; i < 32; ++i) sum += s_sum[i][lane];
    to[h] = sum;
}

cudaError_t forward(const NormArgs &p, int x_dtype, int dtype, cudaStream_t st)
{
    return with_dtype(x_dtype, [&](auto x) { return norm::launch_forward<decltype(x)>(p, dtype, st); });
}

cudaError_t backward(const NormArgs &p, int x_dtype, int dtype, float *dpre, float *dpost, float *dchan, cudaStream_t st)
{
    const int parts = norm_parts(p.T, p.H, heavy_backward(p));
    const cudaError_t e = with_dtype(x_dtype, [&](auto x) { return norm::launch_backward<decltype(x)>(p, dtype, parts, st); });
    if (e != cudaSuccess || (!dpre && !dpost && !dchan)) return e;
    return launch_kernel(norm_parts_kernel, dim3((p.H + 31) / 32, 3), dim3(1024), 0, st, 1, (const float *)p.part, parts, p.H, dpre,
                         dpost, dchan);
}

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

int elem_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

int check_norm(const NormArgs &p, int x_dtype, int dtype)
{
    for (int d : {x_dtype, dtype})
        if (d != MOE_DTYPE_F32 && d != MOE_DTYPE_BF16 && d != MOE_DTYPE_F16) return set_error(MOE_ERR_ARG, "unknown dtype %d", d);
    if (p.T < 0 || p.T > 1 << 24) return set_error(MOE_ERR_SHAPE, "T must be in [0, 2^24] (got %d)", p.T);
    if (p.H < 8 || p.H > kMaxDim || p.H % 8)
        return set_error(MOE_ERR_SHAPE, "H must be a multiple of 8 in [8, %d] (got %d)", kMaxDim, p.H);
    if (p.kind < MOE_GATE_NONE || p.kind > MOE_GATE_FULL) return set_error(MOE_ERR_ARG, "unknown gate kind %d", p.kind);
    if (p.T == 0) return MOE_OK;   // tensors of no rows may be NULL
    if (!p.gate != !p.kind) return set_error(MOE_ERR_ARG, "gate and gate_kind do not agree");
    if (!p.y && (p.gate || p.post)) return set_error(MOE_ERR_ARG, "gate and post_w need y");
    if (p.ldx < p.H || (p.y && p.ldy < p.H)) return set_error(MOE_ERR_SHAPE, "ldx and ldy must be at least H");
    if (p.ldx * elem_bytes(x_dtype) % 16) return set_error(MOE_ERR_ALIGN, "rows of x are not 16-byte aligned (ldx %lld)", p.ldx);
    if (p.y && p.ldy * elem_bytes(dtype) % 16) return set_error(MOE_ERR_ALIGN, "rows of y are not 16-byte aligned (ldy %lld)", p.ldy);
    if (!(p.a - p.a == 0.0f) || !(p.b - p.b == 0.0f)) return set_error(MOE_ERR_ARG, "the scales must be finite");
    for (const void *q : {p.y, (const void *)p.post, (const void *)p.pre})
        if (off(q, 16)) return set_error(MOE_ERR_ALIGN, "y, post_w or pre_w is not 16-byte aligned");
    if (off(p.gate, p.kind == kGateToken ? elem_bytes(dtype) : 16)) return set_error(MOE_ERR_ALIGN, "gate is not aligned");
    return MOE_OK;
}

int done(cudaError_t e, const char *what)
{
    if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return set_error(MOE_OK, "%s", "");
}

}  // namespace

}  // namespace moe

using namespace moe;

#define NORM_PTR(p, a)                                                                                  \
    do {                                                                                                \
        if (!(p)) return set_error(MOE_ERR_ARG, "%s is NULL", #p);                                      \
        if (off((p), (a))) return set_error(MOE_ERR_ALIGN, "%s is not %d-byte aligned", #p, (int)(a));  \
    } while (0)

extern "C" {

size_t moe_block_norm_workspace_size(int T, int H)
{
    if (T < 0 || T > 1 << 24 || H < 8 || H > kMaxDim || H % 8) return 0;
    return 256 + (size_t)norm_parts(T, H, 0) * 3 * H * sizeof(float);
}

int moe_block_norm_forward(const void *x, long long ldx, int x_dtype, const void *y, long long ldy, const void *gate, int gate_kind,
                           int dtype, const float *post_w, const float *pre_w, float eps, float residual_scale,
                           float branch_scale, int T, int H, void *out, void *n, float *kept, void *stream)
{
    NormArgs p = {};
    p.x = x;
    p.y = y;
    p.gate = gate;
    p.ldx = ldx;
    p.ldy = y ? ldy : 0;
    p.post = post_w;
    p.pre = pre_w;
    p.eps = eps;
    p.a = residual_scale;
    p.b = branch_scale;
    p.T = T;
    p.H = H;
    p.kind = gate_kind;
    p.out = out;
    p.n = n;
    p.kept = reinterpret_cast<float2 *>(kept);
    int rc;
    if ((rc = check_norm(p, x_dtype, dtype))) return rc;
    if (!(eps >= 0.0f) || !(eps - eps == 0.0f)) return set_error(MOE_ERR_ARG, "eps must be finite and not negative");
    if (T == 0) return done(cudaSuccess, "");
    if (!n != !pre_w) return set_error(MOE_ERR_ARG, "n and pre_w go together");
    if (!n && !out) return set_error(MOE_ERR_ARG, "out and n are both NULL");
    NORM_PTR(x, 16);
    if (T > 1 && ((out == x && ldx != H) || (n && n == y && ldy != H)))
        return set_error(MOE_ERR_ARG, "out and n are dense: they cannot be an x or y of strided rows");
    if (off(out, 16) || off(n, 16)) return set_error(MOE_ERR_ALIGN, "out or n is not 16-byte aligned");
    if (off(kept, 8)) return set_error(MOE_ERR_ALIGN, "kept is not 8-byte aligned");
    if ((rc = require_device())) return rc;
    return done(forward(p, x_dtype, dtype, (cudaStream_t)stream), "block norm launch");
}

int moe_block_norm_backward(const void *x, long long ldx, int x_dtype, const void *y, long long ldy, const void *gate, int gate_kind,
                            int dtype, const float *post_w, const float *pre_w, const float *kept, float residual_scale,
                            float branch_scale, int T, int H, const void *dout, const void *dn, void *dx, void *dy, void *dgate,
                            float *dpost, float *dpre, void *workspace, size_t workspace_bytes, void *stream)
{
    NormArgs p = {};
    p.x = x;
    p.y = y;
    p.gate = gate;
    p.ldx = ldx;
    p.ldy = y ? ldy : 0;
    p.post = post_w;
    p.pre = pre_w;
    p.a = residual_scale;
    p.b = branch_scale;
    p.T = T;
    p.H = H;
    p.kind = gate_kind;
    p.kept = reinterpret_cast<float2 *>(const_cast<float *>(kept));
    p.dout = dout;
    p.dn = dn;
    p.dx = dx;
    p.dy = dy;
    p.dgate = gate_kind == MOE_GATE_CHANNEL ? nullptr : dgate;
    p.want_post = dpost != nullptr;
    p.want_pre = dpre != nullptr;
    p.want_channel = gate_kind == MOE_GATE_CHANNEL && dgate;
    int rc;
    if ((rc = check_norm(p, x_dtype, dtype))) return rc;
    for (const void *q : {dout, dn, (const void *)dx, (const void *)dy, (const void *)dpost, (const void *)dpre})
        if (off(q, 16)) return set_error(MOE_ERR_ALIGN, "a gradient is not 16-byte aligned");
    if (off(dgate, gate_kind == MOE_GATE_TOKEN ? 4 : 16)) return set_error(MOE_ERR_ALIGN, "dgate is not aligned");
    float *dchan = p.want_channel ? static_cast<float *>(dgate) : nullptr;
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {   // no rows: the sums over them are zero
        if (!dpre && !dpost && !dchan) return done(cudaSuccess, "");
        if ((rc = require_device())) return rc;
        cudaError_t e = cudaSuccess;
        for (float *q : {dpre, dpost, dchan})
            if (q && e == cudaSuccess) e = cudaMemsetAsync(q, 0, (size_t)H * sizeof(float), st);
        return done(e, "block norm backward");
    }
    if (!dn != !pre_w) return set_error(MOE_ERR_ARG, "dn and pre_w go together");
    if (!dn && !dout) return set_error(MOE_ERR_ARG, "dout and dn are both NULL");
    if ((dy && !y) || (dgate && !gate) || (dpost && !post_w) || (dpre && !pre_w))
        return set_error(MOE_ERR_ARG, "a gradient is asked for of an operand that is NULL");
    NORM_PTR(x, 16);
    NORM_PTR(kept, 8);
    if (!workspace) return set_error(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (off(workspace, 256)) return set_error(MOE_ERR_ALIGN, "workspace is not 256-byte aligned");
    const size_t need = moe_block_norm_workspace_size(T, H);
    if (workspace_bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace has %zu bytes; %zu needed", workspace_bytes, need);
    if ((rc = require_device())) return rc;
    p.part = reinterpret_cast<float *>(static_cast<char *>(workspace) + 256);
    p.err = static_cast<int32_t *>(workspace);
    return done(backward(p, x_dtype, dtype, dpre, dpost, dchan, st), "block norm backward launch");
}

}  // extern "C"
