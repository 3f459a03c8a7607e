// block_norm.cuh -- the kernels of the step between two blocks (block_norm.cu has the formulas): arguments, the kernels
// of both directions, and how many CTAs they take.
#pragma once

#include <algorithm>

#include "cluster_wait.cuh"
#include "launch.cuh"
#include "moe_internal.cuh"
#include "vec8.cuh"

namespace moe {
namespace norm {

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

struct RowsShared {
    float sum[2][2][32];   // by turns: a row may exchange once only, and then no barrier stands between its sums' last
                           // read and the next row's
};

// The same on many rows: rows blockIdx, blockIdx + grid, ... on two CTAs an SM or more, so that one works while another
// waits for its warps, the next rows on their way into a ring in shared memory (asynchronous copies; a thread
// reads back only what it copied).  8192 rows of 6144, bf16, full gate: 76 us with the weights in registers (99 with
// them from L1, which the ring leaves too small for them), the kernel above 95.
template <typename X, typename Y, int THREADS>
__global__ void __launch_bounds__(THREADS, 2) norm_rows_kernel(const NormArgs p)
{
    constexpr bool HOLD = THREADS <= 448;   // the weights stay in registers
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ RowsShared sh;
    auto &s_sum = sh.sum;
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

struct BackwardShared {
    uint64_t full[kMaxNormStages];
    float sum[2][4 * 32];
};

// Rows blockIdx, blockIdx + grid, ...; a thread keeps its 8 columns' sums over them.  The rows come through a
// ring in shared memory (one bulk copy an operand), so that the next ones are on their way while one is worked
// on; what is needed again after the row's one exchange between the warps stays in registers.
//
// Beside the memory the issue slots are what is short (8192 rows of 6144, bf16, full gate; 805 MB): two vectors a
// thread on half the warps 177 us (too few warps to fill the slots), the next row's sums beside this row's
// results, formed twice, 211; one vector a thread, with the sums' exchange by its lanes and two conversions an
// instruction 166; what is there known at compile time (KIND, a gate's kind, with the gradients of all that is there;
// -1: whatever is there) 147; the weights asked for ahead of the wait 142.  Without a pre norm 275, known at compile
// time 125.
template <typename X, typename Y, int THREADS, int KIND, bool POST, bool PRE>
__global__ void __launch_bounds__(THREADS) norm_backward_kernel(const NormArgs p)
{
    extern __shared__ __align__(16) uint8_t ring[];
    __shared__ BackwardShared sh;
    auto &full = sh.full;
    auto &s_sum = sh.sum;
    constexpr bool ALL = KIND >= 0;
    const bool has_dout = ALL || p.dout, has_y = ALL || p.y, has_dn = ALL ? PRE : p.dn != nullptr, has_post = ALL ? POST : p.post != nullptr;
    const bool want_dx = ALL || p.dx, want_dy = ALL || p.dy, want_post = ALL ? POST : p.want_post != 0, want_pre = ALL ? PRE : p.want_pre != 0;
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
            if (!ok) {   // nothing more is asked for, and the copies in flight get their time
                atomicOr(p.err, kErrTimeout);
                polls = kSettleLimit;
                uint32_t parity = phase;
                for (int i = 0, at = slot; i < p.stages && row + i * step < p.T; ++i) {
                    poll(&full[at], parity, polls);
                    if (++at == p.stages) {
                        at = 0;
                        parity ^= 1;
                    }
                }
            }
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

inline int norm_threads(int H, int vecs) { return ((H / 8 + vecs - 1) / vecs + 31) / 32 * 32; }

// The backward kernel runs up to 768 threads an SM with 80 registers each: as many CTAs as whole rows fit.  (More of
// them with 72 registers are slower, for what they spill: 6000 rows of 1792, full gate 93 us against 71.)  Rows beyond
// 6144 take 896 threads with 72 registers or 1024 with 64.  So do two rows of 3080 to 4096, which would stand alone,
// where what a thread holds allows it (`heavy`, 0 to 2): both directions of 8192 rows in bf16, two and one, of 3584 without a
// gate 114 us and 138, with a channel's 155 and 156 (fp32 stream 198 and 184), of 4096 without post 110 and 125, without pre
// 101 and 119, with both 140 and 143 (fp32 stream 201 and 195), with a channel's gate too 231 and 164.
// CTAs of one warp: 24 (65536 rows of 256 85 us, with 8 of them 138); of more, 8 (65536 of 512 with 12 155, with 8 150).
inline int ctas_per_sm(int H, int heavy)
{
    const int threads = norm_threads(H, 1);
    if (threads > 384 && threads <= 512) return heavy < (threads <= 448 ? 2 : 1) ? 2 : 1;
    return std::max(1, std::min(threads == 32 ? 24 : 8, 768 / threads));
}

// Its CTAs: as many as stand on 152 SMs, and no more than there are rows for at two each, beyond eight an SM at four
inline int norm_parts(int T, int H, int heavy)
{
    const int ctas = ctas_per_sm(H, heavy), few = 152 * std::min(8, ctas);
    return std::max(1, std::min((T + 1) / 2, std::max(few, std::min((T + 3) / 4, 152 * ctas))));
}

// a post norm and a gate with columns, beside a pre norm
inline int heavy_backward(const NormArgs &p) { return p.dn ? (p.post != nullptr) + (p.kind & 1) : 0; }

// Shared memory of an SM: what rings may take of it, all of it, and what each CTA takes beside its ring and static part
constexpr int kRingBytesSm = 216 * 1024, kSharedBytesSm = 228 * 1024, kCtaBytes = 1024;

// CTAs an SM of the forward kernel with rings of `ring` bytes, by the registers that each bound leaves a thread (72 and
// 64) and by shared memory: a wave and a quarter of them takes two (16384 rows of 1024, fp32 stream, without a gate: 11 CTAs
// 42 us, 12 and a second wave 48)
inline int forward_ctas(int threads, int ring)
{
    const int bytes = (ring + (int)sizeof(RowsShared) + 127) / 128 * 128 + kCtaBytes;
    return std::min((threads <= 448 ? 896 : 1024) / threads, std::min(kRingBytesSm / ring, kSharedBytesSm / bytes));
}

// Rows of `row` bytes in a ring of the backward kernel: what the CTAs of an SM share has to hold all of them, or the last
// ones run as a second wave (65536 rows of 256, bf16, without a gate: rings of 3 rows 56 us, of 4 and a second wave 71;
// 32768 of 768, fp32 stream: 2 rows 87, 3 rows 107).
inline int backward_stages(int row, int parts, int ctas)
{
    const int share = std::min((parts + 151) / 152, ctas);
    const int bytes = kSharedBytesSm / share / 128 * 128 - kCtaBytes - (int)sizeof(BackwardShared);
    return std::max(1, std::min(kMaxNormStages, std::min(kRingBytesSm / share, bytes) / row));
}

// by the stream's type X, one translation unit each (block_norm_f32.cu and so on)
template <typename X>
cudaError_t launch_forward(const NormArgs &p, int dtype, cudaStream_t st);
template <typename X>
cudaError_t launch_backward(NormArgs p, int dtype, int parts, cudaStream_t st);

}  // namespace norm
}  // namespace moe
