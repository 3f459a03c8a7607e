// gated.cu -- the dense gated block in 16 bits, h = silu(x Wg^T) * (x Wu^T), and its gradients:
// launches of the products (kernels: gemm16.cuh, for few tokens gemm_tc.cuh), the elementwise pass between them, and the
// entry points.
//
// With s = sigmoid(g):  dg = dh u s (1 + g (1 - s)),  du = dh g s,
//   dx = dg Wg + du Wu,   dWg = dg^T x,   dWu = du^T x.
//
// Of an element the forward pass keeps A = u s (1 + g (1 - s)) and B = g s for the backward one, so
// that dg = dh A and du = dh B, in 16 bits each (gated_kept.cuh), A in `kept_g` and B in `kept_u`.  The
// other rounding to 16 bits besides the outputs' is that of dg and du, the operands of the
// tensor-core products.  Everything else is fp32.
#include <algorithm>

#include "gemm16.cuh"
#include "tensor_map.cuh"

namespace moe {

namespace {

// fp32 sums, operands bf16 or fp16, `lanes` rows of which `a` is the rows' operand
uint32_t idesc16(int dtype, int lanes, bool a_mn, bool b_mn)
{
    const uint32_t f = dtype == MOE_DTYPE_BF16 ? 1u : 0u;
    return (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) | ((uint32_t)(lanes >> 4) << 24);
}

__device__ __forceinline__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_f(__half v) { return __half2float(v); }
__device__ __forceinline__ void set(__nv_bfloat16 &d, float v) { d = __float2bfloat16_rn(v); }
__device__ __forceinline__ void set(__half &d, float v) { d = __float2half_rn(v); }

// dg, du from dh and the kept factors, 8 values a thread (F is a multiple of 8, so the rows laid end
// to end are).  Bound by memory: 10 bytes a value.
template <typename T, bool FP16>
__global__ void __launch_bounds__(256)
    gated_grad_kernel(const T *__restrict__ dh, const uint16_t *__restrict__ kept_g, const uint16_t *__restrict__ kept_u,
                      long long units, T *__restrict__ dg, T *__restrict__ du)
{
    pdl_wait();
    pdl_launch_dependents();
    const long long i = (long long)blockIdx.x * 256 + threadIdx.x;
    if (i >= units) return;
    union Pack {
        uint4 v;
        T t[8];
    } a, p, q;
    a.v = ld_stream_v4(reinterpret_cast<const uint4 *>(dh) + i);
    const uint4 a4 = ld_stream_v4(reinterpret_cast<const uint4 *>(kept_g) + i), b4 = ld_stream_v4(reinterpret_cast<const uint4 *>(kept_u) + i);
    const uint32_t A[4] = {a4.x, a4.y, a4.z, a4.w}, B[4] = {b4.x, b4.y, b4.z, b4.w};
#pragma unroll
    for (int j = 0; j < 8; ++j) {
        const float d = to_f(a.t[j]);
        set(p.t[j], d * Kept<FP16>::value(j & 1 ? A[j >> 1] : A[j >> 1] << 16));
        set(q.t[j], d * Kept<FP16>::value(j & 1 ? B[j >> 1] : B[j >> 1] << 16));
    }
    reinterpret_cast<uint4 *>(dg)[i] = p.v;
    reinterpret_cast<uint4 *>(du)[i] = q.v;
}

// Few tokens take the kernel with the weights' rows on the lanes, tokens in columns of up to 32: it
// spreads the reduction over clusters, where a pair of SMs walks all of it (about 0.17 us a 64
// inputs); a longer list of columns and short reductions favour the pairs.  Microseconds, few and
// pairs: 6144 x 2048, 1 token 8.0, 18.9, 64 tokens 17.1, 18.9; 2048 x 512, 1 token 4.6, 8.0, 64
// tokens 6.9, 8.0; 1000 x 520, 1 token 4.5, 5.4, 32 tokens 5.9, 5.5; 512 x 512, 8 tokens 4.5, 4.1.
bool few_tokens(int T, int H) { return T <= 16 ? H > 512 : T <= 64 && H >= 2048; }
constexpr int kFewCols = 32;

cudaError_t forward_few(const void *x, long long ldx, const void *wg, const void *wu, int dtype, int T, int H, int F,
                        void *h, void *g, void *u, int32_t *err, cudaStream_t st)
{
    gemm::Maps m;
    cudaError_t e = rows_map(&m.a[0], wg, 16, H, H, F, gemm::kM);
    if (e == cudaSuccess) e = rows_map(&m.a[1], wu, 16, H, H, F, gemm::kM);
    for (int k = 0; 16 * (k + 1) <= kFewCols && e == cudaSuccess; ++k) e = rows_map(&m.b[k], x, 16, H, ldx, T, 16 * (k + 1));
    if (e != cudaSuccess) return e;
    gemm::Args a = {};
    a.E = 1;
    a.rows = T;
    a.M = F;
    a.ksteps = (H + 63) / 64;
    a.out[0] = h;
    a.out[1] = g;
    a.out[2] = u;
    a.ld = F;
    a.dtype = dtype;
    a.idesc = idesc16(dtype, gemm::kM, false, false);
    a.err = err;
    const int mtiles = (F + gemm::kM - 1) / gemm::kM;
    a.split = gemm::choose_split<gemm::kGate, kFewCols, true>(mtiles * ((T + gemm::kSplitCols - 1) / gemm::kSplitCols), a.ksteps);
    a.width = a.split > 1 ? gemm::kSplitCols : kFewCols;
    const int tiles = mtiles * ((T + a.width - 1) / a.width);
    return gemm::launch<gemm::kGate, kFewCols, true>(a, m, std::min(tiles, num_sms() / a.split) * a.split, st);
}

cudaError_t forward(const void *x, long long ldx, const void *wg, const void *wu, int dtype, int T, int H, int F,
                    void *h, void *g, void *u, int32_t *err, cudaStream_t st)
{
    if (few_tokens(T, H)) return forward_few(x, ldx, wg, wu, dtype, T, H, F, h, g, u, err, st);
    gemm16::Args a = {};
    a.rows = T;
    a.cols = F;
    a.groups = 1;
    a.ksteps = a.kphase = (H + 63) / 64;
    a.out[0] = h;
    a.out[1] = g;
    a.out[2] = u;
    a.dtype = dtype;
    a.idesc = idesc16(dtype, 2 * gemm16::kLanes, false, false);
    a.err = err;
    gemm16::plan<gemm16::kGate2>(a);
    gemm16::Maps m;
    cudaError_t e = rows_map(&m.r[0], x, 16, H, ldx, T, a.rbox);
    if (e == cudaSuccess) e = rows_map(&m.c[0], wg, 16, H, H, F, a.width / 2);
    if (e == cudaSuccess) e = rows_map(&m.c[1], wu, 16, H, H, F, a.width / 2);
    return e == cudaSuccess ? gemm16::launch<gemm16::kGate2>(a, m, st) : e;
}

cudaError_t grad_x(const void *dg, const void *du, const void *wg, const void *wu, int dtype, int T, int H, int F,
                   void *dx, int32_t *err, cudaStream_t st)
{
    gemm16::Args a = {};
    a.rows = T;
    a.cols = H;
    a.groups = 1;
    a.kphase = (F + 63) / 64;
    a.ksteps = 2 * a.kphase;
    a.out[0] = dx;
    a.dtype = dtype;
    a.idesc = idesc16(dtype, 2 * gemm16::kLanes, false, true);
    a.err = err;
    gemm16::plan<gemm16::kDx>(a);
    gemm16::Maps m;
    cudaError_t e = rows_map(&m.r[0], dg, 16, F, F, T, a.rbox);
    if (e == cudaSuccess) e = rows_map(&m.r[1], du, 16, F, F, T, a.rbox);
    if (e == cudaSuccess) e = rows_map(&m.c[0], wg, 16, H, H, F, 64);
    if (e == cudaSuccess) e = rows_map(&m.c[1], wu, 16, H, H, F, 64);
    return e == cudaSuccess ? gemm16::launch<gemm16::kDx>(a, m, st) : e;
}

cudaError_t grad_w(const void *dg, const void *du, const void *x, long long ldx, int dtype, int T, int H, int F,
                   void *dwg, void *dwu, int32_t *err, cudaStream_t st)
{
    gemm16::Args a = {};
    a.rows = F;
    a.cols = H;
    a.groups = 2;
    a.ksteps = a.kphase = (T + 63) / 64;
    a.out[0] = dwg;
    a.out[1] = dwu;
    a.dtype = dtype;
    a.idesc = idesc16(dtype, 2 * gemm16::kLanes, true, true);
    a.err = err;
    gemm16::plan<gemm16::kDw>(a);
    gemm16::Maps m;
    cudaError_t e = rows_map(&m.r[0], dg, 16, F, F, T, 64);
    if (e == cudaSuccess) e = rows_map(&m.r[1], du, 16, F, F, T, 64);
    if (e == cudaSuccess) e = rows_map(&m.c[0], x, 16, H, ldx, T, 64);
    return e == cudaSuccess ? gemm16::launch<gemm16::kDw>(a, m, st) : e;
}

constexpr int kMaxGatedDim = 65536, kMaxGatedT = 1 << 24;

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

int check_shape(int dtype, int T, int H, int F, long long ldx)
{
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_error(MOE_ERR_ARG, "dtype must be bf16 or fp16 (got %d)", dtype);
    if (T < 0 || T > kMaxGatedT) return set_error(MOE_ERR_SHAPE, "T must be in [0, 2^24] (got %d)", T);
    if (H < 8 || H > kMaxGatedDim || H % 8)
        return set_error(MOE_ERR_SHAPE, "H must be a multiple of 8 in [8, %d] (got %d)", kMaxGatedDim, H);
    if (F < 8 || F > kMaxGatedDim || F % 8)
        return set_error(MOE_ERR_SHAPE, "F must be a multiple of 8 in [8, %d] (got %d)", kMaxGatedDim, F);
    if (ldx < H) return set_error(MOE_ERR_SHAPE, "ldx must be at least H (got %lld)", ldx);
    if (ldx % 8) return set_error(MOE_ERR_ALIGN, "rows of x are not 16-byte aligned (ldx %lld)", ldx);
    return MOE_OK;
}

#define GATED_PTR(p)                                                                             \
    do {                                                                                         \
        if (!(p)) return set_error(MOE_ERR_ARG, "%s is NULL", #p);                               \
        if (off((p), 16)) return set_error(MOE_ERR_ALIGN, "%s is not 16-byte aligned", #p);      \
    } while (0)

int check_workspace(void *ws, size_t bytes, size_t need)
{
    if (!ws) return set_error(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (off(ws, 256)) return set_error(MOE_ERR_ALIGN, "workspace is not 256-byte aligned");
    if (bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace has %zu bytes; %zu needed", bytes, need);
    return MOE_OK;
}

size_t grad_bytes(int T, int F) { return ((size_t)T * F * 2 + 255) / 256 * 256; }

int done(cudaError_t e, const char *what)
{
    if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return set_error(MOE_OK, "%s", "");
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_gated_workspace_size(int T, int H, int F, int train)
{
    if (T < 0 || T > kMaxGatedT || H < 8 || H > kMaxGatedDim || H % 8 || F < 8 || F > kMaxGatedDim || F % 8) return 0;
    return 256 + (train ? 2 * grad_bytes(T, F) : 0);
}

int moe_gated_forward(const void *x, long long ldx, const void *w_gate, const void *w_up, int dtype, int T, int H, int F,
                      void *h, void *kept_g, void *kept_u, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_shape(dtype, T, H, F, ldx))) return rc;
    if (T == 0) return done(cudaSuccess, "");
    GATED_PTR(x);
    GATED_PTR(w_gate);
    GATED_PTR(w_up);
    GATED_PTR(h);
    if (!kept_g != !kept_u) return set_error(MOE_ERR_ARG, "kept_g and kept_u go together");
    if (off(kept_g, 16) || off(kept_u, 16)) return set_error(MOE_ERR_ALIGN, "kept_g or kept_u is not 16-byte aligned");
    if ((rc = check_workspace(workspace, workspace_bytes, 256)) || (rc = require_device())) return rc;
    return done(forward(x, ldx, w_gate, w_up, dtype, T, H, F, h, kept_g, kept_u, static_cast<int32_t *>(workspace),
                        (cudaStream_t)stream),
                "gated forward launch");
}

int moe_gated_backward(const void *dh, const void *x, long long ldx, const void *w_gate, const void *w_up, const void *kept_g,
                       const void *kept_u, int dtype, int T, int H, int F, void *dx, void *dw_gate, void *dw_up,
                       void *workspace, size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_shape(dtype, T, H, F, ldx))) return rc;
    if (!dw_gate != !dw_up) return set_error(MOE_ERR_ARG, "dw_gate and dw_up go together");
    if (off(dx, 16) || off(dw_gate, 16) || off(dw_up, 16)) return set_error(MOE_ERR_ALIGN, "a gradient is not 16-byte aligned");
    cudaStream_t st = (cudaStream_t)stream;
    if (T == 0) {   // no rows: the weights' gradients are zero
        if (!dw_gate) return done(cudaSuccess, "");
        if ((rc = require_device())) return rc;
        cudaError_t e = cudaMemsetAsync(dw_gate, 0, (size_t)F * H * 2, st);
        if (e == cudaSuccess) e = cudaMemsetAsync(dw_up, 0, (size_t)F * H * 2, st);
        return done(e, "gated backward");
    }
    GATED_PTR(dh);
    GATED_PTR(x);
    GATED_PTR(w_gate);
    GATED_PTR(w_up);
    GATED_PTR(kept_g);
    GATED_PTR(kept_u);
    if ((rc = check_workspace(workspace, workspace_bytes, moe_gated_workspace_size(T, H, F, 1))) || (rc = require_device()))
        return rc;
    if (!dx && !dw_gate) return done(cudaSuccess, "");
    int32_t *err = static_cast<int32_t *>(workspace);
    char *dg = static_cast<char *>(workspace) + 256, *du = dg + grad_bytes(T, F);
    const long long units = (long long)T * F / 8;
    const dim3 grid((unsigned)((units + 255) / 256));
    cudaError_t e =
        dtype == MOE_DTYPE_BF16
            ? launch_kernel(gated_grad_kernel<__nv_bfloat16, false>, grid, dim3(256), 0, st, 1, (const __nv_bfloat16 *)dh,
                            (const uint16_t *)kept_g, (const uint16_t *)kept_u, units, (__nv_bfloat16 *)dg, (__nv_bfloat16 *)du)
            : launch_kernel(gated_grad_kernel<__half, true>, grid, dim3(256), 0, st, 1, (const __half *)dh, (const uint16_t *)kept_g,
                            (const uint16_t *)kept_u, units, (__half *)dg, (__half *)du);
    if (e == cudaSuccess && dx) e = grad_x(dg, du, w_gate, w_up, dtype, T, H, F, dx, err, st);
    if (e == cudaSuccess && dw_gate) e = grad_w(dg, du, x, ldx, dtype, T, H, F, dw_gate, dw_up, err, st);
    return done(e, "gated backward launch");
}

}  // extern "C"
