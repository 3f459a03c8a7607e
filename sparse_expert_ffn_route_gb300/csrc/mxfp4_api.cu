// mxfp4_api.cu -- the extern "C" entry points of the MXFP4 operators: argument checks,
// workspace layout and launches.  See include/moe.h for the contract.
#include "moe_internal.cuh"

namespace moe {

namespace {

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

#define MX_PTR(p, a)                                                                                     \
    do {                                                                                                 \
        if (!(p)) return set_error(MOE_ERR_ARG, "%s is NULL", #p);                                       \
        if (off((p), (a))) return set_error(MOE_ERR_ALIGN, "%s is not %d-byte aligned", #p, (int)(a));   \
    } while (0)

size_t up(size_t v) { return (v + 255) / 256 * 256; }

int check_dtype(int dtype)
{
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_error(MOE_ERR_ARG, "unknown dtype %d", dtype);
    return MOE_OK;
}

int elem_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

constexpr int kMaxMxK = 65536, kMaxMxN = 1 << 20, kMaxMxRows = 1 << 27;

int check_rows(long long rows, int K)
{
    if (rows < 0 || rows > kMaxMxRows) return set_error(MOE_ERR_SHAPE, "rows must be in [0, 2^27] (got %lld)", rows);
    if (K < 32 || K > kMaxMxK || K % 32)
        return set_error(MOE_ERR_SHAPE, "K must be a multiple of 32 in [32, %d] (got %d)", kMaxMxK, K);
    return MOE_OK;
}

int check_workspace(void *ws, size_t bytes, size_t need)
{
    if (!ws) return set_error(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (off(ws, 256)) return set_error(MOE_ERR_ALIGN, "workspace is not 256-byte aligned");
    if (bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace has %zu bytes; %zu needed", bytes, need);
    return MOE_OK;
}

struct FfnLayout {
    size_t x, xs, h, hs, xt, xts, total;
};

// Above this many values of all pairs each token is quantised once and its 4-bit row copied to
// its pairs; below it every pair quantises its token's row, one launch less.  The whole block,
// top-8 of 64 experts, hidden 6144, d_ff 256, microseconds with a quantised row a pair and a token:
// 64 tokens 49.5, 52.5; 170 tokens 64.8, 65.0; 256 tokens 72.7, 66.7; 4096 tokens 524, 350.
constexpr long long kQuantOnce = 1ll << 23;

bool quantise_once(const moe_config &c, long long T) { return c.top_k > 1 && T * c.top_k * c.hidden >= kQuantOnce; }

FfnLayout ffn_layout(const moe_config &c, int T)
{
    const size_t P = (size_t)T * c.top_k;
    FfnLayout L;
    L.x = 256;
    L.xs = L.x + up(P * c.hidden / 2);
    L.h = L.xs + up(P * c.hidden / 32);
    L.hs = L.h + up(P * c.d_ff / 2);
    L.xt = L.hs + up(P * c.d_ff / 32);
    L.xts = L.xt;
    L.total = L.xt;
    if (quantise_once(c, T)) {
        L.xts = L.xt + up((size_t)T * c.hidden / 2);
        L.total = L.xts + up((size_t)T * c.hidden / 32);
    }
    return L;
}

int done(cudaError_t e, const char *what)
{
    if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return set_error(MOE_OK, "%s", "");
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

int moe_quantize_mxfp4(const void *x, int dtype, long long ldx, long long rows, int K, uint8_t *codes, uint8_t *scales,
                       void *stream)
{
    int rc;
    if ((rc = check_dtype(dtype)) || (rc = check_rows(rows, K))) return rc;
    if (ldx < K) return set_error(MOE_ERR_SHAPE, "ldx must be at least K (got %lld)", ldx);
    if (rows == 0) return done(cudaSuccess, "");
    MX_PTR(x, 16);
    if (ldx * elem_bytes(dtype) % 16) return set_error(MOE_ERR_ALIGN, "rows of x are not 16-byte aligned (ldx %lld)", ldx);
    MX_PTR(codes, 16);
    MX_PTR(scales, 16);
    if ((rc = require_device())) return rc;
    return done(launch_quantize_mxfp4(x, dtype, ldx, rows, K, nullptr, nullptr, 0, codes, scales, nullptr,
                                      (cudaStream_t)stream),
                "MXFP4 quantiser launch");
}

int moe_dequantize_mxfp4(const uint8_t *codes, const uint8_t *scales, long long rows, int K, void *y, int dtype,
                         void *stream)
{
    int rc;
    if ((rc = check_dtype(dtype)) || (rc = check_rows(rows, K))) return rc;
    if (rows == 0) return done(cudaSuccess, "");
    MX_PTR(codes, 16);
    MX_PTR(scales, 16);
    MX_PTR(y, 16);
    if ((rc = require_device())) return rc;
    return done(launch_dequantize_mxfp4(codes, scales, rows, K, y, dtype, (cudaStream_t)stream),
                "MXFP4 dequantiser launch");
}

int moe_mxfp4_matmul(const uint8_t *x, const uint8_t *x_scales, int rows, const uint8_t *w, const uint8_t *w_scales,
                     int groups, const int32_t *offsets, int N, int K, void *y, int dtype, void *workspace,
                     size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_dtype(dtype)) || (rc = check_rows(rows, K))) return rc;
    if (N < 1 || N > kMaxMxN) return set_error(MOE_ERR_SHAPE, "N must be in [1, 2^20] (got %d)", N);
    if (groups < 1 || groups > kMaxExperts)
        return set_error(MOE_ERR_SHAPE, "groups must be in [1, %d] (got %d)", kMaxExperts, groups);
    if ((long long)groups * N > kMaxMxRows) return set_error(MOE_ERR_SHAPE, "groups * N must be at most 2^27");
    if (rows == 0) return done(cudaSuccess, "");
    MX_PTR(x, 16);
    MX_PTR(x_scales, 16);
    MX_PTR(w, 16);
    MX_PTR(w_scales, 16);
    MX_PTR(y, 16);
    if (groups > 1 && !offsets) return set_error(MOE_ERR_ARG, "offsets is NULL with %d groups", groups);
    if (off(offsets, 4)) return set_error(MOE_ERR_ALIGN, "offsets is not 4-byte aligned");
    if ((rc = check_workspace(workspace, workspace_bytes, 256)) || (rc = require_device())) return rc;
    return done(launch_mxfp4_matmul(x, x_scales, rows, w, w_scales, groups, offsets, N, K, y, dtype, 0,
                                    static_cast<int32_t *>(workspace), (cudaStream_t)stream),
                "MXFP4 product launch");
}

size_t moe_mxfp4_workspace_size(const moe_config *cfg, int max_tokens)
{
    if (moe_workspace_size(cfg, max_tokens) == 0) return 0;   // the same limits
    return ffn_layout(*cfg, max_tokens).total;
}

int moe_mxfp4_expert_ffn(const moe_config *cfg, const void *x, int x_dtype, int T, const moe_expert_mxfp4 *w,
                         const int32_t *offsets, const int32_t *tok, void *y_pairs, int y_dtype, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = validate_config(cfg, T)) || (rc = check_dtype(x_dtype)) || (rc = check_dtype(y_dtype))) return rc;
    if (T == 0) return done(cudaSuccess, "");
    MX_PTR(x, 16);
    if (!w) return set_error(MOE_ERR_ARG, "weights are NULL");
    MX_PTR(w->w_gate, 16);
    MX_PTR(w->s_gate, 16);
    MX_PTR(w->w_up, 16);
    MX_PTR(w->s_up, 16);
    MX_PTR(w->w_down, 16);
    MX_PTR(w->s_down, 16);
    if (!offsets != !tok) return set_error(MOE_ERR_ARG, "offsets and tok go together");
    if (!offsets && (cfg->n_experts != 1 || cfg->top_k != 1))
        return set_error(MOE_ERR_ARG, "offsets is NULL with %d experts and top_k %d", cfg->n_experts, cfg->top_k);
    if (off(offsets, 4)) return set_error(MOE_ERR_ALIGN, "offsets is not 4-byte aligned");
    if (off(tok, 4)) return set_error(MOE_ERR_ALIGN, "tok is not 4-byte aligned");
    MX_PTR(y_pairs, 16);
    const FfnLayout L = ffn_layout(*cfg, T);
    if ((rc = check_workspace(workspace, workspace_bytes, L.total)) || (rc = require_device())) return rc;
    cudaStream_t st = (cudaStream_t)stream;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    int32_t *err = static_cast<int32_t *>(workspace);
    const int E = cfg->n_experts, H = cfg->hidden, F = cfg->d_ff, P = T * cfg->top_k;
    // The quantiser waits for what the stream held before the call before it lets the next kernel
    // start, so that the two products may read weights and lists early.
    const int32_t *limit = offsets ? offsets + E : nullptr;
    cudaError_t e;
    if (tok && quantise_once(*cfg, T)) {
        e = launch_quantize_mxfp4(x, x_dtype, H, T, H, nullptr, nullptr, 0, ws + L.xt, ws + L.xts, err, st);
        if (e == cudaSuccess)
            e = launch_gather_mxfp4(ws + L.xt, ws + L.xts, P, H, tok, limit, T, ws + L.x, ws + L.xs, err, st);
    } else {
        e = launch_quantize_mxfp4(x, x_dtype, H, P, H, tok, limit, T, ws + L.x, ws + L.xs, err, st);
    }
    if (e == cudaSuccess)
        e = launch_mxfp4_gate_up(ws + L.x, ws + L.xs, P, w->w_gate, w->s_gate, w->w_up, w->s_up, E, offsets, F, H,
                                 ws + L.h, ws + L.hs, 1, err, st);
    if (e == cudaSuccess)
        e = launch_mxfp4_matmul(ws + L.h, ws + L.hs, P, w->w_down, w->s_down, E, offsets, H, F, y_pairs, y_dtype, 1, err, st);
    return done(e, "MXFP4 expert FFN launch");
}

}  // extern "C"
