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
#include <algorithm>

#include "cluster_wait.cuh"
#include "launch.cuh"
#include "moe_internal.cuh"
#include "vec8.cuh"

namespace moe {

namespace {

enum Gate { kGateNone = MOE_GATE_NONE, kGateChannel = MOE_GATE_CHANNEL, kGateToken = MOE_GATE_TOKEN, kGateFull = MOE_GATE_FULL };

constexpr int kMaxNormThreads = 512;   // a row of kMaxDim in two vectors of 8 a thread
constexpr int kVecs = 2;
constexpr int kMaxNormStages = 4;

struct NormArgs {
    const void *x, *y, *gate;
    long long ldx, ldy;
    const float *post, *pre;
    float eps, a, b;
    int T, H, kind;
    void *out, *n;
    float2 *kept;
    // backward
    const void *dout, *dn;
    void *dx, *dy, *dgate;
    float *part;               // [parts][3][H]: this CTA's sums for dpre, dpost and a channel's gate
    int want_post, want_pre, want_channel;
    int stages;                // rows of the ring
    int32_t *err;
};

// sums of N values over the block, in every thread; `s` holds N floats a warp and is not used again before
// the next barrier
template <int N>
__device__ __forceinline__ void block_sums(float (&v)[N], float *s)
{
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += __shfl_xor_sync(0xffffffffu, v[i], off);
    const int warps = blockDim.x >> 5;
    if (warps == 1) return;
    if ((threadIdx.x & 31) == 0)
#pragma unroll
        for (int i = 0; i < N; ++i) s[(threadIdx.x >> 5) * N + i] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 0.0f;
    for (int w = 0; w < warps; ++w)
#pragma unroll
        for (int i = 0; i < N; ++i) v[i] += s[w * N + i];
}

__device__ __forceinline__ float inverse(float sum, int H, float eps)
{
    const float ms = sum / (float)H + eps;
    return ms == 0.0f ? 0.0f : 1.0f / sqrtf(ms);   // a row of zeros stays one; NaN stays NaN
}

// One row a CTA, kVecs vectors of 8 a thread, held in registers between the passes over the row.
template <typename X, typename Y>
__global__ void __launch_bounds__(kMaxNormThreads) norm_forward_kernel(const NormArgs p)
{
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float s_sum[2][kMaxNormThreads / 32];
    const size_t t = blockIdx.x;
    const X *x = static_cast<const X *>(p.x) + t * p.ldx;
    const Y *y = static_cast<const Y *>(p.y) + t * p.ldy;
    const Y *gate = static_cast<const Y *>(p.gate) + (p.kind == kGateFull ? t * p.H : 0);
    Vec8<X> vx[kVecs];
    Vec8<Y> vy[kVecs], vg[kVecs];
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int h = (v * blockDim.x + threadIdx.x) * 8;
        vx[v].zero();
        vy[v].zero();
        if (h < p.H) {
            vx[v].load(x + h);
            if (p.y) vy[v].load(y + h);
            if (p.kind & 1) vg[v].load(gate + h);   // a channel's or an element's
        }
    }
    const float row_gate = p.kind == kGateToken ? to_f32(static_cast<const Y *>(p.gate)[t]) : 1.0f;
    float iy = 1.0f;
    if (p.post) {
        float ss[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kVecs; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(vy[v].get(i), vy[v].get(i), ss[0]);
        block_sums(ss, s_sum[0]);
        iy = inverse(ss[0], p.H, p.eps);
    }
    const float scale = p.b * row_gate;
    float o[kVecs][8], ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int h = (v * blockDim.x + threadIdx.x) * 8;
        Vec8<float> w;
        if (p.post && h < p.H) w.load(p.post + h);
        Vec8<X> r;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            o[v][i] = p.a * vx[v].get(i);
            if (p.y) {
                float z = vy[v].get(i);
                if (p.post) z = z * iy * w.get(i);
                if (p.kind & 1) z *= vg[v].get(i);
                o[v][i] = fmaf(scale, z, o[v][i]);
            }
            if (h < p.H) ss[0] = fmaf(o[v][i], o[v][i], ss[0]);
            r.set(i, o[v][i]);
        }
        if (p.out && h < p.H) r.store(static_cast<X *>(p.out) + t * p.H + h);
    }
    float io = 1.0f;
    if (p.pre) {
        block_sums(ss, s_sum[1]);
        io = inverse(ss[0], p.H, p.eps);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int h = (v * blockDim.x + threadIdx.x) * 8;
            if (h >= p.H) continue;
            Vec8<float> w;
            w.load(p.pre + h);
            Vec8<Y> r;
#pragma unroll
            for (int i = 0; i < 8; ++i) r.set(i, o[v][i] * io * w.get(i));
            r.store(static_cast<Y *>(p.n) + t * p.H + h);
        }
    }
    if (p.kept && threadIdx.x == 0) p.kept[t] = make_float2(iy, io);
}

// bytes of a row of each operand in the ring, in the order x, dout, y, dn, full gate; 0: absent
struct RowBytes {
    uint32_t x, dout, y, dn, gate;
    __host__ __device__ RowBytes(const NormArgs &p, int ex, int ey)
    {
        x = p.H * ex;
        dout = p.dout ? p.H * ex : 0;
        y = p.y ? p.H * ey : 0;
        dn = p.dn ? p.H * ey : 0;
        gate = p.kind == kGateFull ? p.H * ey : 0;
    }
    __host__ __device__ uint32_t total() const { return x + dout + y + dn + gate; }
};

// Rows blockIdx, blockIdx + grid, ...; a thread keeps its columns' sums over them.  The rows come through a
// ring in shared memory (one bulk copy an operand), so that the next ones are on their way during the one
// exchange between the warps that a row needs, and the row is read twice from there.
template <typename X, typename Y>
__global__ void __launch_bounds__(kMaxNormThreads) norm_backward_kernel(const NormArgs p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t full[kMaxNormStages];
    __shared__ float s_sum[2][3 * (kMaxNormThreads / 32)];
    const RowBytes rb(p, sizeof(X), sizeof(Y));
    const uint32_t stage = rb.total();
    const int tid = threadIdx.x;
    if (tid == 0) {
        for (int i = 0; i < p.stages; ++i) mbar_init(&full[i], 1);
        fence_mbar_init();
    }
    __syncthreads();
    pdl_wait();
    pdl_launch_dependents();
    const auto fetch = [&](int row, int slot) {   // by thread 0
        if (row >= p.T) return;
        const size_t t = row;
        uint8_t *to = ring + (size_t)slot * stage;
        mbar_arrive_expect_tx(&full[slot], stage);
        const auto copy = [&](const void *from, size_t at, uint32_t bytes) {
            if (!bytes) return;
            bulk_g2s(to, static_cast<const uint8_t *>(from) + at, bytes, &full[slot]);
            to += bytes;
        };
        copy(p.x, t * p.ldx * sizeof(X), rb.x);
        copy(p.dout, t * rb.dout, rb.dout);
        copy(p.y, t * p.ldy * sizeof(Y), rb.y);
        copy(p.dn, t * rb.dn, rb.dn);
        copy(p.gate, t * rb.gate, rb.gate);
    };
    if (tid == 0)
        for (int i = 0; i < p.stages; ++i) fetch(blockIdx.x + i * gridDim.x, i);

    float dpre[kVecs][8], dpost[kVecs][8], dchan[kVecs][8];
#pragma unroll
    for (int v = 0; v < kVecs; ++v)
#pragma unroll
        for (int i = 0; i < 8; ++i) dpre[v][i] = dpost[v][i] = dchan[v][i] = 0.0f;
    const float inv_h = 1.0f / (float)p.H;
    bool ok = true;
    int turn = 0, slot = 0;
    uint32_t phase = 0;
    float2 next_kept = make_float2(0.0f, 0.0f);
    float next_gate = 1.0f;
    const auto numbers = [&](int row) {   // of a row, asked for one row ahead
        if (row >= p.T) return;
        next_kept = p.kept[row];
        if (p.kind == kGateToken) next_gate = to_f32(static_cast<const Y *>(p.gate)[row]);
    };
    numbers(blockIdx.x);
    for (int row = blockIdx.x, prev = -1; row < p.T; row += gridDim.x, turn ^= 1) {
        const size_t t = row;
        const float iy = next_kept.x, io = next_kept.y, row_gate = next_gate, scale = p.b * row_gate;
        numbers(row + gridDim.x);
        if (ok) {
            int polls = kClusterWaitLimit;
            poll(&full[slot], phase, polls);
            ok = polls > 0;
            if (!ok) atomicOr(p.err, kErrTimeout);
        }
        const uint8_t *sx = ring + (size_t)slot * stage, *so = sx + rb.x, *sy = so + rb.dout, *sn = sy + rb.y, *sg = sn + rb.dn;
        // What is absent reads as what leaves the formulas as they are: y, dn, dout 0, weights and gate 1.
        const auto operands = [&](int h, Vec8<Y> &y, Vec8<Y> &g, Vec8<float> &post) {
            if (p.y) y.load(reinterpret_cast<const Y *>(sy) + h);
            else y.zero();
            if (p.kind == kGateFull) g.load(reinterpret_cast<const Y *>(sg) + h);
            else if (p.kind == kGateChannel) g.load(static_cast<const Y *>(p.gate) + h);
            else g.fill(1.0f);
            if (p.post) post.load(p.post + h);
            else post.fill(1.0f);
        };
        float o[kVecs][8], e[kVecs][8], s[3] = {0.0f, 0.0f, 0.0f};   // sum w out, sum q e, sum q out
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int h = (v * blockDim.x + tid) * 8;
            if (h >= p.H) continue;
            Vec8<X> x, dout;
            Vec8<Y> y, g, dn;
            Vec8<float> post, pre;
            operands(h, y, g, post);
            x.load(reinterpret_cast<const X *>(sx) + h);
            if (p.dout) dout.load(reinterpret_cast<const X *>(so) + h);
            else dout.zero();
            if (p.dn) {
                dn.load(reinterpret_cast<const Y *>(sn) + h);
                pre.load(p.pre + h);
            } else {
                dn.zero();
                pre.fill(1.0f);
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float q = y.get(i) * post.get(i) * g.get(i), w = dn.get(i) * pre.get(i);
                o[v][i] = fmaf(scale * iy, q, p.a * x.get(i));
                e[v][i] = fmaf(io, w, dout.get(i));
                s[0] = fmaf(w, o[v][i], s[0]);
                s[1] = fmaf(q, e[v][i], s[1]);
                s[2] = fmaf(q, o[v][i], s[2]);
            }
        }
        block_sums(s, s_sum[turn]);   // (its barrier: the row before this one has been read by all)
        if (tid == 0 && prev >= 0 && ok && p.stages > 1) fetch(prev + p.stages * gridDim.x, slot == 0 ? p.stages - 1 : slot - 1);
        const float k = io * s[0] * inv_h * io * io;         // (io^3 alone would leave fp32's range)
        const float qd = s[1] - k * s[2];                    // sum q d
        const float c2 = p.post ? iy * qd * inv_h * iy * scale : 0.0f;
        if (p.kind == kGateToken && p.dgate && tid == 0) static_cast<float *>(p.dgate)[t] = p.b * iy * qd;
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int h = (v * blockDim.x + tid) * 8;
            if (h >= p.H) continue;
            Vec8<X> rx;
            Vec8<Y> y, g, dn, ry, rg;
            Vec8<float> post;
            operands(h, y, g, post);
            if (p.dn) dn.load(reinterpret_cast<const Y *>(sn) + h);
            else dn.zero();
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float d = fmaf(-k, o[v][i], e[v][i]), yi = y.get(i) * iy;
                const float bd = p.b * d, dz = bd * row_gate * g.get(i), dg = bd * yi * post.get(i);
                rx.set(i, p.a * d);
                rg.set(i, dg);
                dchan[v][i] += dg;
                dpost[v][i] = fmaf(dz, yi, dpost[v][i]);
                dpre[v][i] = fmaf(dn.get(i), o[v][i] * io, dpre[v][i]);
                ry.set(i, iy * fmaf(dz, post.get(i), -c2 * y.get(i)));
            }
            if (p.dx) rx.store(static_cast<X *>(p.dx) + t * p.H + h);
            if (p.dy) ry.store(static_cast<Y *>(p.dy) + t * p.H + h);
            if (p.kind == kGateFull && p.dgate) rg.store(static_cast<Y *>(p.dgate) + t * p.H + h);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");   // these reads come before the next copy into the slot
        prev = row;
        if (++slot == p.stages) {
            slot = 0;
            phase ^= 1;
        }
        if (p.stages == 1) {
            __syncthreads();
            if (tid == 0 && ok) fetch(row + gridDim.x, 0);
        }
    }
    if (!ok) {   // what is still in flight gets its time
        int polls = kSettleLimit;
        poll(&full[slot], phase, polls);
    }
    float *part = p.part + (size_t)blockIdx.x * 3 * p.H;
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int h = (v * blockDim.x + tid) * 8;
        if (h >= p.H) continue;
        Vec8<float> r;
        const auto put = [&](const float (&sum)[8], int which) {
#pragma unroll
            for (int i = 0; i < 8; ++i) r.set(i, sum[i]);
            r.store(part + (size_t)which * p.H + h);
        };
        if (p.want_pre) put(dpre[v], 0);
        if (p.want_post) put(dpost[v], 1);
        if (p.want_channel) put(dchan[v], 2);
    }
}

// Sums of the CTAs' parts, 32 columns a CTA, in a fixed order.
__global__ void __launch_bounds__(512) norm_parts_kernel(const float *part, int parts, int H, float *dpre, float *dpost, float *dchan)
{
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float s_sum[16][32];
    float *to = blockIdx.y == 0 ? dpre : blockIdx.y == 1 ? dpost : dchan;
    if (!to) return;
    const int lane = threadIdx.x & 31, w = threadIdx.x >> 5, h = blockIdx.x * 32 + lane;
    float sum = 0.0f;
    if (h < H)
        for (int i = w; i < parts; i += 16) sum += part[((size_t)i * 3 + blockIdx.y) * H + h];
    s_sum[w][lane] = sum;
    __syncthreads();
    if (w || h >= H) return;
    for (int i = 1; i < 16; ++i) sum += s_sum[i][lane];
    to[h] = sum;
}

int norm_threads(int H) { return ((H / 8 + kVecs - 1) / kVecs + 31) / 32 * 32; }

// CTAs of the backward kernel: those of 128 registers a thread that fit 152 SMs, and no more than there are
// rows for at four each
int norm_parts(int T, int H) { return std::max(1, std::min((T + 3) / 4, 152 * std::min(8, kMaxNormThreads / norm_threads(H)))); }

cudaError_t launch_forward(const NormArgs &p, int x_dtype, int dtype, cudaStream_t st)
{
    return with_dtype(x_dtype, [&](auto xt) {
        return with_dtype(dtype, [&](auto yt) {
            return launch_kernel(norm_forward_kernel<decltype(xt), decltype(yt)>, dim3(p.T), dim3(norm_threads(p.H)), 0, st, 1, p);
        });
    });
}

constexpr int kRingBytesSm = 216 * 1024;   // shared memory of an SM for rings

cudaError_t launch_backward(NormArgs p, int x_dtype, int dtype, float *dpre, float *dpost, float *dchan, cudaStream_t st)
{
    const int parts = norm_parts(p.T, p.H), threads = norm_threads(p.H);
    const cudaError_t e = with_dtype(x_dtype, [&](auto xt) {
        return with_dtype(dtype, [&](auto yt) {
            using X = decltype(xt);
            using Y = decltype(yt);
            const int row = (int)RowBytes(p, sizeof(X), sizeof(Y)).total();
            const int ctas = std::max(1, std::min((parts + 151) / 152, kMaxNormThreads / threads));
            p.stages = std::max(1, std::min(kMaxNormStages, kRingBytesSm / ctas / row));
            return launch_kernel(norm_backward_kernel<X, Y>, dim3(parts), dim3(threads), (size_t)p.stages * row, st, 1, p);
        });
    });
    if (e != cudaSuccess || (!dpre && !dpost && !dchan)) return e;
    return launch_kernel(norm_parts_kernel, dim3((p.H + 31) / 32, 3), dim3(512), 0, st, 1, (const float *)p.part, parts, p.H, dpre,
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
    return 256 + (size_t)norm_parts(T, H) * 3 * H * sizeof(float);
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
    if (off(out, 16) || off(n, 16)) return set_error(MOE_ERR_ALIGN, "out or n is not 16-byte aligned");
    if (off(kept, 8)) return set_error(MOE_ERR_ALIGN, "kept is not 8-byte aligned");
    if ((rc = require_device())) return rc;
    return done(launch_forward(p, x_dtype, dtype, (cudaStream_t)stream), "block norm launch");
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
    return done(launch_backward(p, x_dtype, dtype, dpre, dpost, dchan, st), "block norm backward launch");
}

}  // extern "C"
