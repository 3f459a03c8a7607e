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
constexpr int kMaxNormStages = 4;   // backward
constexpr int kRowStages = 3;       // forward

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

// Sums of N (a power of two, at most 4) values a thread over the block, in every thread.  `s` holds 32 floats for
// each and is not used again before the next barrier; `fence` runs before the barrier.
template <int N, typename F>
__device__ __forceinline__ void block_sums(float (&v)[N], float *s, F &&fence)
{
    const int lane = threadIdx.x & 31, warps = blockDim.x >> 5;
    constexpr int each = 32 / N;   // lanes that end with one value's sum
    ReduceScatter<N, 16>::run(v, lane);
    if (warps > 1) {
        if (lane % each == 0) s[lane / each * 32 + (threadIdx.x >> 5)] = v[0];
        fence();
        __syncthreads();
        // lanes of value n add up the warps' sums of n, `each` at a time
        const float *from = s + lane / each * 32;
        float sum = 0.0f;
        for (int w = lane % each; w < warps; w += each) sum += from[w];
#pragma unroll
        for (int off = each / 2; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
        v[0] = sum;
    } else {
        fence();
        __syncwarp();
    }
    const float mine = v[0];
#pragma unroll
    for (int n = 0; n < N; ++n) v[n] = __shfl_sync(0xffffffffu, mine, n * each);
}

// eight values into shared memory, asynchronously
template <typename T>
__device__ __forceinline__ void copy8(T *to, const T *from)
{
#pragma unroll
    for (int i = 0; i < 8; i += 16 / (int)sizeof(T)) cp_async16(to + i, from + i, true);
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
    __shared__ float s_sum[2][32];
    const auto nothing = [] {};
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
        for (int v = 0; v < kVecs; ++v) {
            float y[8];
            vy[v].get(y);
#pragma unroll
            for (int i = 0; i < 8; ++i) ss[0] = fmaf(y[i], y[i], ss[0]);
        }
        block_sums(ss, s_sum[0], nothing);
        iy = inverse(ss[0], p.H, p.eps);
    }
    const float scale = p.b * row_gate * iy;
    float o[kVecs][8], ss[1] = {0.0f};
#pragma unroll
    for (int v = 0; v < kVecs; ++v) {
        const int h = (v * blockDim.x + threadIdx.x) * 8;
        if (h >= p.H) continue;
        vx[v].get(o[v]);
#pragma unroll
        for (int i = 0; i < 8; ++i) o[v][i] *= p.a;
        if (p.y) {
            float z[8], f[8];
            vy[v].get(z);
            if (p.post) {
                Vec8<float> w;
                w.load(p.post + h);
                w.get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= f[i];
            }
            if (p.kind & 1) {
                vg[v].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) z[i] *= f[i];
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) o[v][i] = fmaf(scale, z[i], o[v][i]);
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) ss[0] = fmaf(o[v][i], o[v][i], ss[0]);
        if (p.out) {
            Vec8<X> r;
            r.set(o[v]);
            r.store(static_cast<X *>(p.out) + t * p.H + h);
        }
    }
    float io = 1.0f;
    if (p.pre) {
        block_sums(ss, s_sum[1], nothing);
        io = inverse(ss[0], p.H, p.eps);
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int h = (v * blockDim.x + threadIdx.x) * 8;
            if (h >= p.H) continue;
            Vec8<float> w;
            float f[8];
            w.load(p.pre + h);
            w.get(f);
#pragma unroll
            for (int i = 0; i < 8; ++i) f[i] *= o[v][i] * io;
            Vec8<Y> r;
            r.set(f);
            r.store(static_cast<Y *>(p.n) + t * p.H + h);
        }
    }
    if (p.kept && threadIdx.x == 0) p.kept[t] = make_float2(iy, io);
}

// The same on many rows: rows blockIdx, blockIdx + grid, ... on two CTAs an SM, so that one works while the other
// waits for its warps, the next rows on their way into a ring in shared memory (asynchronous copies; a thread
// reads back only what it copied).  8192 rows of 6144, bf16, full gate: 76 us with the weights in registers (99 with
// them from L1, which the ring leaves too small for them), the kernel above 95.
template <typename X, typename Y, int THREADS>
__global__ void __launch_bounds__(THREADS, 2) norm_rows_kernel(const NormArgs p)
{
    constexpr bool HOLD = THREADS <= 448;   // the weights stay in registers
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ float s_sum[2][2][32];   // by turns: a row may exchange once only, and then no barrier stands between its
                                        // sums' last read and the next row's
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t bx = p.H * sizeof(X), by = p.y ? p.H * sizeof(Y) : 0, bg = p.kind == kGateFull ? p.H * sizeof(Y) : 0;
    const uint32_t stage = bx + by + bg;
    const int tid = threadIdx.x, step = gridDim.x;
    const auto nothing = [] {};
    float next_gate = 1.0f;
    const auto fetch = [&](int row, uint8_t *to) {
        if (row < p.T) {
            const size_t t = row;
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int h = (v * blockDim.x + tid) * 8;
                if (h >= p.H) continue;
                copy8(reinterpret_cast<X *>(to) + h, static_cast<const X *>(p.x) + t * p.ldx + h);
                if (by) copy8(reinterpret_cast<Y *>(to + bx) + h, static_cast<const Y *>(p.y) + t * p.ldy + h);
                if (bg) copy8(reinterpret_cast<Y *>(to + bx + by) + h, static_cast<const Y *>(p.gate) + t * p.H + h);
            }
        }
        cp_async_commit();
    };
    const auto number = [&](int row) {
        if (p.kind == kGateToken && row < p.T) next_gate = to_f32(static_cast<const Y *>(p.gate)[row]);
    };
    for (int i = 0; i < kRowStages - 1; ++i) fetch(blockIdx.x + i * step, ring + (size_t)i * stage);
    number(blockIdx.x);
    Vec8<float> wpost[kVecs], wpre[kVecs];
    const auto weights = [&] {
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int h = (v * blockDim.x + tid) * 8;
            if (p.post && h < p.H) wpost[v].load(p.post + h);
            if (p.pre && h < p.H) wpre[v].load(p.pre + h);
        }
    };
    if (HOLD) weights();
    int slot = 0, last = kRowStages - 1, turn = 0;
    for (int row = blockIdx.x; row < p.T; row += step, turn ^= 1) {
        const size_t t = row;
        const float row_gate = next_gate;
        number(row + step);
        fetch(row + (kRowStages - 1) * step, ring + (size_t)last * stage);
        cp_async_wait<kRowStages - 1>();
        const uint8_t *sx = ring + (size_t)slot * stage, *sy = sx + bx, *sg = sy + by;
        last = slot;
        slot = slot + 1 == kRowStages ? 0 : slot + 1;
        float z[kVecs][8], iy = 1.0f;
        if (p.y) {
            float ss[1] = {0.0f};
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int h = (v * blockDim.x + tid) * 8;
                if (h >= p.H) continue;
                Vec8<Y> y;
                y.load(reinterpret_cast<const Y *>(sy) + h);
                y.get(z[v]);
#pragma unroll
                for (int i = 0; i < 8; ++i) ss[0] = fmaf(z[v][i], z[v][i], ss[0]);
            }
            if (p.post) {
                block_sums(ss, s_sum[turn][0], nothing);
                iy = inverse(ss[0], p.H, p.eps);
            }
        }
        const float scale = p.b * row_gate * iy;
        float ss[1] = {0.0f};
#pragma unroll
        for (int v = 0; v < kVecs; ++v) {
            const int h = (v * blockDim.x + tid) * 8;
            if (h >= p.H) continue;
            float o[8], f[8];
            Vec8<X> x;
            x.load(reinterpret_cast<const X *>(sx) + h);
            x.get(o);
            if (p.y) {
                if (p.post) {
                    if (!HOLD) wpost[v].load(p.post + h);
                    wpost[v].get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[v][i] *= f[i];
                }
                if (p.kind & 1) {
                    Vec8<Y> g;
                    if (bg) g.load(reinterpret_cast<const Y *>(sg) + h);
                    else g.load(static_cast<const Y *>(p.gate) + h);
                    g.get(f);
#pragma unroll
                    for (int i = 0; i < 8; ++i) z[v][i] *= f[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] = fmaf(scale, z[v][i], p.a * o[i]);
            } else {
#pragma unroll
                for (int i = 0; i < 8; ++i) o[i] *= p.a;
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                ss[0] = fmaf(o[i], o[i], ss[0]);
                z[v][i] = o[i];
            }
            if (p.out) {
                Vec8<X> r;
                r.set(o);
                r.store(static_cast<X *>(p.out) + t * p.H + h);
            }
        }
        float io = 1.0f;
        if (p.pre) {
            block_sums(ss, s_sum[turn][1], nothing);
            io = inverse(ss[0], p.H, p.eps);
#pragma unroll
            for (int v = 0; v < kVecs; ++v) {
                const int h = (v * blockDim.x + tid) * 8;
                if (h >= p.H) continue;
                float f[8];
                if (!HOLD) wpre[v].load(p.pre + h);
                wpre[v].get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) f[i] *= z[v][i] * io;
                Vec8<Y> r;
                r.set(f);
                r.store(static_cast<Y *>(p.n) + t * p.H + h);
            }
        }
        if (p.kept && tid == 0) p.kept[t] = make_float2(iy, io);
    }
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

// Rows blockIdx, blockIdx + grid, ...; a thread keeps its 8 columns' sums over them.  The rows come through a
// ring in shared memory (one bulk copy an operand), so that the next ones are on their way while one is worked
// on; what is needed again after the row's one exchange between the warps stays in registers.
//
// Beside the memory the issue slots are what is short (8192 rows of 6144, bf16, full gate; 805 MB): two vectors a
// thread on half the warps 177 us (too few warps to fill the slots), the next row's sums beside this row's
// results, formed twice, 211; one vector a thread, with the sums' exchange by its lanes and two conversions an
// instruction 166; what is there known at compile time (KIND, a gate's kind with all operands and
// gradients; -1: whatever is there) 147; the weights asked for ahead of the wait 142.
template <typename X, typename Y, int THREADS, int KIND>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const NormArgs p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ uint64_t full[kMaxNormStages];
    __shared__ float s_sum[2][4 * 32];
    constexpr bool ALL = KIND >= 0;
    const bool has_dout = ALL || p.dout, has_y = ALL || p.y, has_dn = ALL || p.dn, has_post = ALL || p.post;
    const bool want_dx = ALL || p.dx, want_dy = ALL || p.dy, want_post = ALL || p.want_post, want_pre = ALL || p.want_pre;
    const int kind = ALL ? KIND : p.kind;
    const bool vector = kind & 1, want_channel = ALL ? KIND == kGateChannel : p.want_channel;
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

    float dpre[8], dpost[8], dchan[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) dpre[i] = dpost[i] = dchan[i] = 0.0f;
    const float inv_h = 1.0f / (float)p.H;
    const int h = tid * 8, step = gridDim.x;
    const bool on = h < p.H;
    float2 next_kept = make_float2(0.0f, 0.0f);
    float next_gate = 1.0f;
    const auto numbers = [&](int row) {   // of a row, asked for one row ahead
        if (row >= p.T) return;
        next_kept = p.kept[row];
        if (kind == kGateToken) next_gate = to_f32(static_cast<const Y *>(p.gate)[row]);
    };
    numbers(blockIdx.x);
    bool ok = true;
    int turn = 0, slot = 0;
    uint32_t phase = 0;
    for (int row = blockIdx.x; row < p.T; row += step, turn ^= 1) {
        const size_t t = row;
        const float iy = next_kept.x, io = next_kept.y, row_gate = next_gate, scale = p.b * row_gate;
        numbers(row + step);
        Vec8<float> wpost, wpre;   // asked for ahead of the wait: the ring leaves L1 too small to keep them
        if (on && has_post) wpost.load(p.post + h);
        if (on && has_dn) wpre.load(p.pre + h);
        if (ok) {
            int polls = kClusterWaitLimit;
            poll(&full[slot], phase, polls);
            ok = polls > 0;
            if (!ok) atomicOr(p.err, kErrTimeout);
        }
        const uint8_t *sx = ring + (size_t)slot * stage, *so = sx + rb.x, *sy = so + rb.dout, *sn = sy + rb.y, *sg = sn + rb.dn;
        // What is absent reads as what leaves the formulas as they are: y, dn, dout 0, weights and gate 1.
        Vec8<Y> vy, vg, vn;
        float o[8], e[8], s[4] = {0.0f, 0.0f, 0.0f, 0.0f};   // sum w out, sum q e, sum q out
        if (on) {
            Vec8<X> vx, vd;
            float f[8], q[8];
            vx.load(reinterpret_cast<const X *>(sx) + h);
            vx.get(o);
            if (has_dout) vd.load(reinterpret_cast<const X *>(so) + h);
            else vd.zero();
            vd.get(e);
            if (has_y) vy.load(reinterpret_cast<const Y *>(sy) + h);
            else vy.zero();
            vy.get(q);
            if (has_post) {
                wpost.get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] *= f[i];
            }
            if (vector) {
                vg.load(kind == kGateFull ? reinterpret_cast<const Y *>(sg) + h : static_cast<const Y *>(p.gate) + h);
                vg.get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) q[i] *= f[i];
            } else {
                vg.fill(1.0f);
            }
            const float by = scale * iy;
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] = fmaf(by, q[i], p.a * o[i]);
            if (has_dn) {
                vn.load(reinterpret_cast<const Y *>(sn) + h);
                float w[8];
                vn.get(w);
                wpre.get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    w[i] *= f[i];
                    e[i] = fmaf(io, w[i], e[i]);
                    s[0] = fmaf(w[i], o[i], s[0]);
                }
            } else {
                vn.zero();
            }
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                s[1] = fmaf(q[i], e[i], s[1]);
                s[2] = fmaf(q[i], o[i], s[2]);
            }
        }
        block_sums(s, s_sum[turn], [] { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); });   // reads come before the next copy
        if (tid == 0 && ok) fetch(row + p.stages * step, slot);
        const float k = io * s[0] * inv_h * io * io;         // (io^3 alone would leave fp32's range)
        const float qd = s[1] - k * s[2];                    // sum q d
        const float c2 = has_post ? iy * qd * inv_h * iy * scale * iy : 0.0f;
        if (kind == kGateToken && p.dgate && tid == 0) static_cast<float *>(p.dgate)[t] = p.b * iy * qd;
        if (on) {
            float d[8], y[8], g[8], f[8], r[8];
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                d[i] = fmaf(-k, o[i], e[i]);
                r[i] = p.a * d[i];
                d[i] *= p.b;
            }
            if (want_dx) {
                Vec8<X> v;
                v.set(r);
                v.store(static_cast<X *>(p.dx) + t * p.H + h);
            }
            if (has_dn) {
                vn.get(f);
#pragma unroll
                for (int i = 0; i < 8; ++i) dpre[i] = fmaf(f[i], o[i] * io, dpre[i]);
            }
            if (has_y) {
                float unit[8];
                vy.get(y);
                vg.get(g);
                if (has_post) {
                    wpost.get(unit);
#pragma unroll
                    for (int i = 0; i < 8; ++i) unit[i] *= iy;
                } else {
#pragma unroll
                    for (int i = 0; i < 8; ++i) unit[i] = 1.0f;
                }
                if (vector) {
#pragma unroll
                    for (int i = 0; i < 8; ++i) r[i] = d[i] * y[i] * unit[i];   // the gate's gradient
                    if (kind == kGateFull && p.dgate) {
                        Vec8<Y> v;
                        v.set(r);
                        v.store(static_cast<Y *>(p.dgate) + t * p.H + h);
                    }
                    if (want_channel)
#pragma unroll
                        for (int i = 0; i < 8; ++i) dchan[i] += r[i];
                }
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    d[i] *= vector ? g[i] : row_gate;   // dz
                    r[i] = fmaf(d[i], unit[i], -c2 * y[i]);
                }
                if (want_post)
#pragma unroll
                    for (int i = 0; i < 8; ++i) dpost[i] = fmaf(d[i], y[i] * iy, dpost[i]);
                if (want_dy) {
                    Vec8<Y> v;
                    v.set(r);
                    v.store(static_cast<Y *>(p.dy) + t * p.H + h);
                }
            }
        }
        if (++slot == p.stages) {
            slot = 0;
            phase ^= 1;
        }
    }
    if (!ok) {   // what is still in flight gets its time
        int polls = kSettleLimit;
        poll(&full[slot], phase, polls);
    }
    if (!on) return;
    float *part = p.part + (size_t)blockIdx.x * 3 * p.H + h;
    const auto put = [&](const float (&sum)[8], int which) {
        Vec8<float> r;
        r.set(sum);
        r.store(part + (size_t)which * p.H);
    };
    if (want_pre) put(dpre, 0);
    if (want_post) put(dpost, 1);
    if (want_channel) put(dchan, 2);
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
#pragma unroll 4
        for (int i = w; i < parts; i += 16) sum += part[((size_t)i * 3 + blockIdx.y) * H + h];
    s_sum[w][lane] = sum;
    __syncthreads();
    if (w || h >= H) return;
    for (int i = 1; i < 16; ++i) sum += s_sum[i][lane];
    to[h] = sum;
}

int norm_threads(int H, int vecs) { return ((H / 8 + vecs - 1) / vecs + 31) / 32 * 32; }

// CTAs of the backward kernel: as many as stand on 152 SMs by their registers (up to 768 threads an SM), and no
// more than there are rows for at two each
constexpr int kGradThreads = 768;
int ctas_per_sm(int H) { return std::max(1, std::min(8, kGradThreads / norm_threads(H, 1))); }
int norm_parts(int T, int H) { return std::max(1, std::min((T + 1) / 2, 152 * ctas_per_sm(H))); }

constexpr int kRingBytesSm = 216 * 1024;   // shared memory of an SM for rings

cudaError_t launch_forward(const NormArgs &p, int x_dtype, int dtype, cudaStream_t st)
{
    const int threads = norm_threads(p.H, kVecs);
    return with_dtype(x_dtype, [&](auto xt) {
        return with_dtype(dtype, [&](auto yt) {
            using X = decltype(xt);
            using Y = decltype(yt);
            const int ring = kRowStages * p.H * (int)(sizeof(X) + (p.y ? sizeof(Y) : 0) + (p.kind == kGateFull ? sizeof(Y) : 0));
            const int fit = std::min(2 * kMaxNormThreads / threads, kRingBytesSm / ring);   // CTAs of an SM
            // (three rows a CTA fill its ring; with fewer the kernel of one row a CTA begins sooner)
            if (fit >= 2 && p.T >= 3 * fit * num_sms())
                return launch_kernel(threads <= 448 ? norm_rows_kernel<X, Y, 448> : norm_rows_kernel<X, Y, 512>, dim3(fit * num_sms()),
                                     dim3(threads), ring, st, 1, p);
            return launch_kernel(norm_forward_kernel<X, Y>, dim3(p.T), dim3(threads), 0, st, 1, p);
        });
    });
}

cudaError_t launch_backward(NormArgs p, int x_dtype, int dtype, float *dpre, float *dpost, float *dchan, cudaStream_t st)
{
    const int parts = norm_parts(p.T, p.H), threads = norm_threads(p.H, 1);
    const cudaError_t e = with_dtype(x_dtype, [&](auto xt) {
        return with_dtype(dtype, [&](auto yt) {
            using X = decltype(xt);
            using Y = decltype(yt);
            const int row = (int)RowBytes(p, sizeof(X), sizeof(Y)).total();
            p.stages = std::max(1, std::min(kMaxNormStages, kRingBytesSm / std::min((parts + 151) / 152, ctas_per_sm(p.H)) / row));
            const auto go = [&](auto kind) {
                constexpr int KIND = decltype(kind)::value;
                // 80, 72 and 64 registers a thread
                return launch_kernel(threads <= kGradThreads ? norm_backward_kernel<X, Y, kGradThreads, KIND>
                                     : threads <= 896        ? norm_backward_kernel<X, Y, 896, KIND>
                                                             : norm_backward_kernel<X, Y, 1024, KIND>,
                                     dim3(parts), dim3(threads), (size_t)p.stages * row, st, 1, p);
            };
            using std::integral_constant;
            const bool all = p.dout && p.y && p.dn && p.post && p.dx && p.dy && p.want_post && p.want_pre;
            if (all && p.kind == kGateNone) return go(integral_constant<int, kGateNone>());
            if (all && p.kind == kGateChannel && p.want_channel) return go(integral_constant<int, kGateChannel>());
            if (all && p.kind == kGateToken && p.dgate) return go(integral_constant<int, kGateToken>());
            if (all && p.kind == kGateFull && p.dgate) return go(integral_constant<int, kGateFull>());
            return go(integral_constant<int, -1>());
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
