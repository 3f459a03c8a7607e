// balance.cu -- how evenly a batch's routing loads the experts, and the gradient of the router's logits.
//
// Of sequence s with L counted tokens and c[s][e] kept pairs of expert e, C = sum_e c, and the router's scores
// sig = 1 / (1 + exp(-l)) normalised to p = sig / sum_e sig:
//   f[s][e] = E c[s][e] / C,  P[s][e] = sum_t p / L,  loss = mean over sequences with L > 0 of sum_e f P.
// (One for an even load; f counts and has no gradient.)  Backward, with G_e = dloss f / (L n) and the
// applied weights w_i = scale g_i / sum_j g_j, g_i = sig of the kept expert i:
//   dl_e  = (G_e - sum_j G_j p_j) p_e (1 - sig_e)
//   dl_i += scale h_i (1 - sig_i) (dw_i - sum_j h_j dw_j),  h = g / sum g
//           (without norm_topk_prob: scale sig_i (1 - sig_i) dw_i).
//
// Scores far below zero are taken relative to the largest, t = exp(l - m) / (1 + exp(l)), so that p keeps its
// digits where every sig is a denormal number or zero.
//
// A warp holds a token's row, or several narrow ones at once.  Both directions are one read of the logits: bound by
// memory for the widths of a router (256 fp32 logits are 1 KB a token), for narrower ones by the instructions a token.
#include <algorithm>

#include "launch.cuh"
#include "moe_internal.cuh"
#include "vec8.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8, kLossWarps = 16;
constexpr int kMaxChunks = 608;      // four CTAs an SM
constexpr int kMinChunk = 2 * kWarps;   // tokens
constexpr int grad_ctas(int per) { return per >= 12 ? 3 : 4; }   // CTAs an SM of the gradient's kernel, by its registers
// Parts of a chunk are one warp's each where they have fewer tokens than this in the mean (30 sequences of one token,
// 221 experts: 9.5 us, by the block 19.3; 2000 sequences of ten, 128 experts: by a warp each 4 us slower)
constexpr int kShortPart = 4;
constexpr int kMaxSequences = 1 << 20;
static_assert(kMaxTopK <= 16, "a row's lanes hold its places");

struct BalanceArgs {
    const void *logits;
    long long ld;
    const int32_t *ids, *keff, *offsets;
    const uint8_t *valid;
    int T, E, K, S, chunk;
    int finish;        // the kernel of the chunks forms the loss too
    // sums of a chunk's part of a sequence, in slot (chunk + sequence): a later part has a later chunk or
    // a later sequence, so no two share a slot and a sequence's are consecutive
    float *psum;       // [slots][E]
    int32_t *pcount;   // [slots][E]
    int32_t *pmeta;    // [slots][2] counted tokens, kept pairs
    float *ploss;      // [S][blocks of 32 experts]
    float *loss;
    int32_t *counts, *tokens;
    int32_t *err, *ticket;
    // backward
    const float *dloss, *dw;
    void *dlogits;
    float scale;
    int norm;
};

constexpr float kNegInf = -__builtin_huge_valf();

// A lane's part of a row that G lanes of a warp share: VEC 4 takes groups of four consecutive logits, VEC 1 every G'th one.
template <int VEC, int G>
__device__ __forceinline__ int expert_of(int j, int lane)
{
    return VEC == 4 ? ((j >> 2) * G + lane) * 4 + (j & 3) : j * G + lane;
}

// the lanes of a warp that share this lane's row
template <int G>
__device__ __forceinline__ unsigned row_lanes()
{
    return G == 32 ? 0xffffffffu : ((1u << (G % 32)) - 1) << (threadIdx.x % 32 / G * G);
}

// The same over G lanes each; the whole warp comes here.
template <int G>
__device__ __forceinline__ bool any_of(bool v)
{
    return G == 32 ? __any_sync(0xffffffffu, v) : (__ballot_sync(0xffffffffu, v) & row_lanes<G>()) != 0;
}

template <int G = 32>
__device__ __forceinline__ float sum_of(float v)
{
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(0xffffffffu, v, off);
    return v;
}

template <int G>
__device__ __forceinline__ float max_of(float v)
{
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(0xffffffffu, v, off));
    return v;
}

// a row as it lies in memory, so that the next token's is on its way while one is worked on
template <typename T, int PER, int VEC, int G>
struct RawRow {
    union __align__(16) {
        uint2 w[PER * sizeof(T) / 8];
        T t[PER];
    };
    __device__ __forceinline__ RawRow()   // (what a row does not reach is never loaded, and scores 0)
    {
#pragma unroll
        for (int j = 0; j < PER; ++j) from_f32(t[j], kNegInf);
    }
    __device__ __forceinline__ void load(const T *row, int E, int lane)
    {
#pragma unroll
        for (int j = 0; j < PER; j += VEC) {
            const int e = expert_of<VEC, G>(j, lane);
            if (e >= E) continue;
            if constexpr (VEC == 1) t[j] = row[e];
            else if constexpr (sizeof(T) == 4) *reinterpret_cast<uint4 *>(t + j) = *reinterpret_cast<const uint4 *>(row + e);
            else *reinterpret_cast<uint2 *>(t + j) = *reinterpret_cast<const uint2 *>(row + e);
        }
    }
    __device__ __forceinline__ void get(float (&l)[PER]) const
    {
#pragma unroll
        for (int j = 0; j < PER; j += 2) pair_to_f32(t + j, l[j], l[j + 1]);
    }
};

constexpr float kLow = -60.0f;   // sums of scores above exp(-60) are far from fp32's smallest numbers
constexpr float kLog2e = 1.44269504f;

__device__ __forceinline__ float ex2(float v)
{
    float r;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

__device__ __forceinline__ float rcp(float v)
{
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(v));
    return r;
}

// sig = 1 / (1 + q) and 1 - sig = q sig with q = exp(-l).  (Where q has left fp32's range sig is 0, and so is what is
// formed here of 1 - sig, which only stands in products with sig.)
__device__ __forceinline__ void sigmoid(float l, float &sig, float &rest)
{
    const float q = ex2(-kLog2e * l);
    sig = rcp(1.0f + q);
    rest = sig * fminf(q, 3.0e38f);
}

// f(j, score, 1 - sig) for the row's N logits of this lane, the scores up to a common factor; a row of nothing but
// -inf scores 0.
template <typename T, int PER, int VEC, int G, typename F>
__device__ __forceinline__ void scores(const RawRow<T, PER, VEC, G> &raw, F &&f)
{
    float l[PER];
    raw.get(l);
    bool high = false;
#pragma unroll
    for (int j = 0; j < PER; ++j) high |= l[j] > kLow;
    high = any_of<G>(high);
    if (G == 32 ? high : __all_sync(0xffffffffu, high)) {
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            float v, rest;
            sigmoid(l[j], v, rest);
            f(j, v, rest);
        }
        return;
    }
    float m = kNegInf;
#pragma unroll
    for (int j = 0; j < PER; ++j) m = fmaxf(m, l[j]);
    m = max_of<G>(m);
#pragma unroll
    for (int j = 0; j < PER; ++j) {
        float v, rest;
        sigmoid(l[j], v, rest);
        if (!high) {   // (1 + exp(l) is 1; NaN stays)
            v = l[j] == kNegInf ? 0.0f : expf(l[j] - m);
            rest = 1.0f;
        }
        f(j, v, rest);
    }
}

// the last sequence that begins at or before token t (or the first), by G lanes
template <int G>
__device__ __forceinline__ int sequence_of(const int32_t *offsets, int S, int t, int lane)
{
    int s = 0, n = S;   // it lies in [s, s + n)
    while (n > 1) {
        const int step = (n + G - 1) / G, at = lane * step;
        const int got = max(1, __popc(__ballot_sync(row_lanes<G>(), at < n && offsets[s + at] <= t)));
        n = min(step, n - (got - 1) * step);
        s += (got - 1) * step;
    }
    return s;
}

// the slots of a sequence's sums (none where its offsets are wrong: false)
__device__ __forceinline__ bool slots_of(const BalanceArgs &p, int s, int &first, int &last)
{
    const int lo = p.offsets[s], hi = p.offsets[s + 1];
    first = 0;
    last = -1;
    if (lo < 0 || lo > hi || hi > p.T) return false;
    if (lo < hi) {
        first = lo / p.chunk + s;
        last = (hi - 1) / p.chunk + s;
    }
    return true;
}

// by one thread, at the very end
__device__ __forceinline__ void put_loss(const BalanceArgs &p, float total, int used, bool wrong)
{
    if (wrong) atomicOr(p.err, kErrBadOffsets);
    p.loss[0] = wrong ? __int_as_float(0x7fc00000) : used ? total / (float)used : 0.0f;
    *p.ticket = 0;
}

// place k of token t, counted if it is kept: 1, or 0
__device__ __forceinline__ int count_pair(const BalanceArgs &p, int t, int k, int *count)
{
    const int kept = p.keff[t], e = p.ids[(size_t)t * p.K + k];
    if (k == 0 && (kept < 0 || kept > p.K)) atomicOr(p.err, kErrBadKeff);
    if (k >= kept) return 0;
    if (e < 0 || e >= p.E) {
        atomicOr(p.err, kErrBadExpertId);
        return 0;
    }
    atomicAdd(&count[e], 1);
    return 1;
}

// the sums of a warp's groups, in the lanes of the first
template <int PER, int G>
__device__ __forceinline__ void add_groups(float (&sum)[PER])
{
#pragma unroll
    for (int off = G; off < 32; off *= 2)
#pragma unroll
        for (int j = 0; j < PER; ++j) sum[j] += __shfl_xor_sync(0xffffffffu, sum[j], off);
}

// The parts [first, last] of a chunk, each by one warp, its rows the only ones on their way: many short sequences.
// `count` holds a warp's counts.
template <typename T, int PER, int VEC, int G>
__device__ __forceinline__ void short_parts(const BalanceArgs &p, int first, int last, int begin, int end, RawRow<T, PER, VEC, G> &raw,
                                            int *count)
{
    const int warp = threadIdx.x / 32, wl = threadIdx.x % 32, lane = wl % G;
    const T *logits = static_cast<const T *>(p.logits);
    int left = end - begin;   // sequences in order have no more tokens here; with others the loss is NaN, and this ends
    // (a lane looks at one of 32 sequences of the warp's, most of which may be empty)
    for (int s0 = first + warp; s0 <= last; s0 += 32 * kWarps) {
        const int my = s0 + wl * kWarps;
        int my_lo = 0, my_hi = 0;
        if (my <= last) {
            my_lo = max(p.offsets[my], begin);
            my_hi = min(p.offsets[my + 1], end);
        }
        for (unsigned some = __ballot_sync(0xffffffffu, my_lo < my_hi); some; some &= some - 1) {
            const int which = __ffs(some) - 1, lo = __shfl_sync(0xffffffffu, my_lo, which), hi = __shfl_sync(0xffffffffu, my_hi, which);
            if ((left -= hi - lo) < 0) return;
            for (int e = wl; e < p.E; e += 32) count[e] = 0;
            __syncwarp();
            float sum[PER];
#pragma unroll
            for (int j = 0; j < PER; ++j) sum[j] = 0.0f;
            int counted = 0, pairs = 0;
            for (int t0 = lo; t0 < hi; t0 += 32 / G) {
                const int t = t0 + wl / G;
                const bool on = t < hi && (!p.valid || p.valid[t]);
                if (G == 32 && !on) continue;
                if (t < hi) raw.load(logits + (size_t)t * p.ld, p.E, lane);
                counted += on && lane == 0;
                if (on && lane < p.K) pairs += count_pair(p, t, lane, count);
                float v[PER], total = 0.0f;
                scores(raw, [&](int j, float score, float) {
                    v[j] = score;
                    total += score;
                });
                total = sum_of<G>(total);
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                if (on)
#pragma unroll
                    for (int j = 0; j < PER; ++j) sum[j] = fmaf(v[j], inv, sum[j]);
            }
            pairs = __reduce_add_sync(0xffffffffu, pairs);
            counted = __reduce_add_sync(0xffffffffu, counted);
            add_groups<PER, G>(sum);
            __syncwarp();
            const size_t slot = (size_t)blockIdx.x + s0 + which * kWarps;
            for (int e = wl; e < p.E; e += 32) p.pcount[slot * p.E + e] = count[e];
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int e = expert_of<VEC, G>(j, lane);
                if (wl < G && e < p.E) p.psum[slot * p.E + e] = sum[j];
            }
            if (wl < 2) p.pmeta[slot * 2 + wl] = wl ? pairs : counted;
            __syncwarp();
        }
    }
}

template <typename T, int PER, int VEC, int G>
__global__ void __launch_bounds__(32 * kWarps, 4) balance_parts_kernel(const BalanceArgs p)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int R = 32 / G;     // rows of a warp
    __shared__ float s_sum[kWarps][kMaxExperts];
    __shared__ int s_count[kMaxExperts], s_meta[2], s_last;
    const int tid = threadIdx.x, wl = tid & 31, warp = tid >> 5, lane = wl % G, group = wl / G;
    const int begin = blockIdx.x * p.chunk, end = min(p.T, begin + p.chunk);
    RawRow<T, PER, VEC, G> raw;      // of token t0 + group, this warp's next
    const T *logits = static_cast<const T *>(p.logits);
    const auto fetch = [&](int t) {
        if (t < end) raw.load(logits + (size_t)t * p.ld, p.E, lane);
    };
    int t0 = begin + warp * R;
    fetch(t0 + group);
    const int first_seq = sequence_of<32>(p.offsets, p.S, begin, wl), last_seq = sequence_of<32>(p.offsets, p.S, end - 1, wl);
    const bool many = (last_seq - first_seq) * kShortPart > end - begin;
    if (many) short_parts<T, PER, VEC, G>(p, first_seq, last_seq, begin, end, raw, reinterpret_cast<int *>(s_sum[warp]));
    for (int e = tid; e < p.E; e += 32 * kWarps) s_count[e] = 0;
    if (tid < 2) s_meta[tid] = 0;
    __syncthreads();
    for (int s = first_seq; s <= last_seq && !many; ++s) {
        const int lo = max(p.offsets[s], begin), hi = min(p.offsets[s + 1], end);
        if (p.offsets[s] >= end) break;
        if (lo >= hi) continue;
        float sum[PER];
#pragma unroll
        for (int j = 0; j < PER; ++j) sum[j] = 0.0f;
        int counted = 0;
        while (t0 < hi) {
            const int t = t0 + group;
            const bool on = lo <= t && t < hi && (!p.valid || p.valid[t]);
            float v[PER], total = 0.0f;
            scores(raw, [&](int j, float score, float) {
                v[j] = score;
                total += score;
            });
            const bool over = R == 1 || t0 + R <= hi || hi == end;   // (else the next sequence has the rest of these rows)
            if (over) {
                t0 += kWarps * R;
                fetch(t0 + group);
            }
            if (R > 1 || on) {
                total = sum_of<G>(total);
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                if (on) {
                    ++counted;
#pragma unroll
                    for (int j = 0; j < PER; ++j) sum[j] = fmaf(v[j], inv, sum[j]);
                }
            }
            if (!over) break;
        }
        int pairs = 0;
        for (int i = tid; i < (hi - lo) * p.K; i += 32 * kWarps) {
            const int at = lo + i / p.K;
            if (!p.valid || p.valid[at]) pairs += count_pair(p, at, i % p.K, s_count);
        }
        add_groups<PER, G>(sum);
#pragma unroll
        for (int j = 0; j < PER; ++j) {
            const int e = expert_of<VEC, G>(j, lane);
            if (group == 0 && e < p.E) s_sum[warp][e] = sum[j];
        }
        if (lane == 0 && counted) atomicAdd(&s_meta[0], counted);
        if (pairs) atomicAdd(&s_meta[1], pairs);
        __syncthreads();
        const size_t slot = (size_t)blockIdx.x + s;
        for (int e = tid; e < p.E; e += 32 * kWarps) {
            float v = s_sum[0][e];
#pragma unroll
            for (int w = 1; w < kWarps; ++w) v += s_sum[w][e];
            p.psum[slot * p.E + e] = v;
            p.pcount[slot * p.E + e] = s_count[e];
            s_count[e] = 0;
        }
        if (tid < 2) {
            p.pmeta[slot * 2 + tid] = s_meta[tid];
            s_meta[tid] = 0;
        }
        __syncthreads();
    }
    if (!p.finish) return;
    // few sums: the last CTA adds them up, a sequence a warp
    if (tid == 0) {
        __threadfence();
        s_last = atomicAdd(p.ticket, 1) == (int)gridDim.x - 1;
    }
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    float total = 0.0f;
    int used = 0;
    bool wrong = false;
    for (int s = warp; s < p.S; s += kWarps) {
        int first, last;
        wrong |= !slots_of(p, s, first, last);
        int tokens = 0, pairs = 0;
        for (int i = first + wl; i <= last; i += 32) {
            tokens += __ldcg(p.pmeta + 2 * i);
            pairs += __ldcg(p.pmeta + 2 * i + 1);
        }
        tokens = __reduce_add_sync(0xffffffffu, tokens);
        pairs = __reduce_add_sync(0xffffffffu, pairs);
        if (wl == 0) p.tokens[s] = tokens;
        used += tokens > 0;
        const float even = pairs > 0 ? (float)p.E / ((float)pairs * (float)max(tokens, 1)) : 0.0f;
        for (int e = wl; e < p.E; e += 32) {
            float sum = 0.0f;
            int count = 0;
#pragma unroll 4
            for (int i = first; i <= last; ++i) {
                sum += __ldcg(p.psum + (size_t)i * p.E + e);
                count += __ldcg(p.pcount + (size_t)i * p.E + e);
            }
            p.counts[(size_t)s * p.E + e] = count;
            total = fmaf((float)count * even, sum, total);
        }
    }
    total = sum_of(total);
    if (tid < 2) s_meta[tid] = 0;
    __syncthreads();
    if (wl == 0) {
        s_sum[0][warp] = total;
        if (used) atomicAdd(&s_meta[0], used);
        if (wrong) atomicOr(&s_meta[1], 1);
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) total += s_sum[0][w];
        put_loss(p, total, s_meta[0], s_meta[1] != 0);
    }
}

// A sequence's sums for 32 experts a CTA; the last CTA adds up the loss.
__global__ void __launch_bounds__(32 * kLossWarps) balance_loss_kernel(const BalanceArgs p)
{
    pdl_wait();
    pdl_launch_dependents();
    __shared__ float s_sum[kLossWarps][32];
    __shared__ int s_count[kLossWarps][32], s_meta[2], s_last, s_used, s_bad;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, warps = blockDim.x >> 5;
    const int s = blockIdx.x, e = blockIdx.y * 32 + lane;
    if (tid < 2) s_meta[tid] = 0;
    __syncthreads();
    int first, last;
    slots_of(p, s, first, last);
    float sum = 0.0f;
    int count = 0, meta[2] = {0, 0};
    if (e < p.E)
#pragma unroll 4
        for (int i = first + warp; i <= last; i += warps) {
            sum += p.psum[(size_t)i * p.E + e];
            count += p.pcount[(size_t)i * p.E + e];
        }
    for (int i = first + tid; i <= last; i += blockDim.x) {
        meta[0] += p.pmeta[2 * i];
        meta[1] += p.pmeta[2 * i + 1];
    }
    s_sum[warp][lane] = sum;
    s_count[warp][lane] = count;
    if (meta[0]) atomicAdd(&s_meta[0], meta[0]);
    if (meta[1]) atomicAdd(&s_meta[1], meta[1]);
    __syncthreads();
    if (warp == 0) {
        for (int w = 1; w < warps; ++w) {
            sum += s_sum[w][lane];
            count += s_count[w][lane];
        }
        if (e < p.E) p.counts[(size_t)s * p.E + e] = count;
        const int tokens = s_meta[0], pairs = s_meta[1];
        float part = e < p.E && pairs > 0 ? (float)count * ((float)p.E / (float)pairs) * (sum / (float)max(tokens, 1)) : 0.0f;
        part = sum_of(part);
        if (lane == 0) {
            p.ploss[(size_t)s * gridDim.y + blockIdx.y] = part;
            if (blockIdx.y == 0) p.tokens[s] = tokens;
            __threadfence();
            s_last = atomicAdd(p.ticket, 1) == (int)(gridDim.x * gridDim.y) - 1;
        }
    }
    if (tid == 0) s_used = s_bad = 0;
    __syncthreads();
    if (!s_last) return;
    __threadfence();
    int used = 0, wrong = 0;
    for (int i = tid; i < p.S; i += blockDim.x) {
        used += __ldcg(p.tokens + i) > 0;
        wrong |= p.offsets[i] < 0 || p.offsets[i] > p.offsets[i + 1] || p.offsets[i + 1] > p.T;
    }
    float total = 0.0f;
    for (long long i = tid; i < (long long)p.S * gridDim.y; i += blockDim.x) total += __ldcg(p.ploss + i);
    total = sum_of(total);
    if (lane == 0) s_sum[0][warp] = total;
    if (used) atomicAdd(&s_used, used);
    if (wrong) atomicOr(&s_bad, 1);
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < warps; ++w) total += s_sum[0][w];
        put_loss(p, total, s_used, s_bad != 0);
    }
}

template <typename T, typename D, int PER, int VEC, int G>
__global__ void __launch_bounds__(32 * kWarps, grad_ctas(PER)) balance_backward_kernel(const BalanceArgs p)
{
    pdl_wait();
    pdl_launch_dependents();
    constexpr int R = 32 / G;     // rows of a warp
    constexpr unsigned ALL = 0xffffffffu;
    __shared__ __align__(16) float s_add[kWarps][R * PER * G];
    __shared__ uint8_t s_mark[kWarps][R * PER * G];
    __shared__ int s_used;
    const int tid = threadIdx.x, wl = tid & 31, warp = tid >> 5, lane = wl % G, group = wl / G;
    float *add = s_add[warp] + group * PER * G;
    uint8_t *mark = s_mark[warp] + group * PER * G;
    const int begin = blockIdx.x * p.chunk, end = min(p.T, begin + p.chunk);
    const T *logits = static_cast<const T *>(p.logits);
    // of the next token: its row, and on the lanes below K its places
    RawRow<T, PER, VEC, G> raw;
    int next_id = -1, next_keff = 0;
    float next_dw = 0.0f;
    const auto fetch = [&](int t) {
        if (t >= end) return;
        raw.load(logits + (size_t)t * p.ld, p.E, lane);
        if (p.dw) {
            next_keff = p.keff[t];
            if (lane < p.K) {
                next_id = p.ids[(size_t)t * p.K + lane];
                next_dw = p.dw[(size_t)t * p.K + lane];
            }
        }
    };
    int t0 = begin + warp * R;
    fetch(t0 + group);
    if (tid == 0) s_used = 0;
    if (p.dw)
#pragma unroll
        for (int j = 0; j < PER; ++j) add[j * G + lane] = 0.0f;
    __syncthreads();
    if (p.dloss) {
        int used = 0;
        for (int i = tid; i < p.S; i += 32 * kWarps) used += p.tokens[i] > 0;
        used = __reduce_add_sync(ALL, used);
        if (wl == 0 && used) atomicAdd(&s_used, used);
        __syncthreads();
    }
    int s = sequence_of<G>(p.offsets, p.S, begin, lane), have = -1;
    int from = p.offsets[s], to = p.offsets[s + 1];
    float slope[PER];
#pragma unroll
    for (int j = 0; j < PER; ++j) slope[j] = 0.0f;
    for (; t0 < end; t0 += kWarps * R) {
        const int t = t0 + group;
        if (to <= t && t < end && s + 1 < p.S) {
            s = sequence_of<G>(p.offsets, p.S, t, lane);
            from = p.offsets[s];
            to = p.offsets[s + 1];
        }
        const bool inside = t < end && from <= t && t < to && !(p.valid && !p.valid[t]);
        const bool some = R == 1 ? inside : __any_sync(ALL, inside);
        float d[PER], total = 0.0f, dot = 0.0f;
        const int keff = next_keff, id = lane < min(keff, p.K) ? next_id : -1;
        const float my_dw = next_dw;
        const bool on = inside && p.dw && id >= 0 && id < p.E;
        const float mine = on ? to_f32(logits[(size_t)t * p.ld + id]) : kNegInf;   // (in L1)
        if (on) mark[id] = (uint8_t)lane;
        if (some && p.dloss) {
            if (inside && s != have) {   // G of another sequence
                have = s;
                int pairs = 0;
#pragma unroll
                for (int j = 0; j < PER; ++j) {
                    const int e = expert_of<VEC, G>(j, lane), c = e < p.E ? p.counts[(size_t)s * p.E + e] : 0;
                    pairs += c;
                    slope[j] = (float)c;
                }
                pairs = __reduce_add_sync(row_lanes<G>(), pairs);
                const float each = pairs > 0 ? p.dloss[0] * ((float)p.E / (float)pairs) / ((float)max(p.tokens[s], 1) * (float)max(s_used, 1)) : 0.0f;
#pragma unroll
                for (int j = 0; j < PER; ++j) slope[j] *= each;
            }
            __syncwarp();
            scores(raw, [&](int j, float v, float rest) {
                total += v;
                dot = fmaf(v, slope[j], dot);
                d[j] = v * rest;
            });
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) d[j] = 0.0f;
        }
        fetch(t + kWarps * R);
        if (some) {
            const float dw = on ? my_dw : 0.0f;
            float g = 0.0f, r = 0.0f;
            if (p.dw) {
                if (inside && lane < min(keff, p.K) && !on) atomicOr(p.err, kErrBadExpertId);
                if (inside && (keff < 0 || keff > p.K)) atomicOr(p.err, kErrBadKeff);
                sigmoid(mine, g, r);
                if (p.norm) {
                    const bool high = any_of<G>(mine > kLow);
                    if (!(R == 1 ? high : __all_sync(ALL, high))) {
                        const float m = max_of<G>(mine);
                        if (!high) {
                            g = mine == kNegInf ? 0.0f : expf(mine - m);
                            r = 1.0f;
                        }
                    }
                }
            }
            __syncwarp();   // (the marks)
            // the token's four sums at once
            constexpr int each = G / 4;   // lanes that end with one
            float sums[4] = {total, dot, g, g * dw};
            ReduceScatter<4, G / 2>::run(sums, lane);
            total = __shfl_sync(ALL, sums[0], 0, G);
            if (p.dloss) {
                const float inv = total == 0.0f ? 0.0f : 1.0f / total;
                dot = __shfl_sync(ALL, sums[0], each, G) * inv;
#pragma unroll
                for (int j = 0; j < PER; ++j) d[j] *= (slope[j] - dot) * inv;
            }
            if (p.dw) {
                float val;
                if (p.norm) {
                    const float sum = __shfl_sync(ALL, sums[0], 2 * each, G), inv = sum == 0.0f ? 0.0f : 1.0f / sum;
                    val = p.scale * g * inv * r * (dw - __shfl_sync(ALL, sums[0], 3 * each, G) * inv);
                } else {
                    const float q = __expf(-fabsf(mine)), one = rcp(1.0f + q);   // sig (1 - sig), the same for l and -l
                    val = p.scale * q * one * one * dw;
                }
                if (__all_sync(ALL, !on || mark[id] == lane)) {   // (a comparison of the lanes' ids takes twice the time of all this)
                    if (on) add[id] = val;
                } else {   // an expert kept twice: in order of its places
                    for (int i = 0; i < p.K; ++i) {
                        if (lane == i && on) add[id] += val;
                        __syncwarp();
                    }
                }
                __syncwarp();
#pragma unroll
                for (int j = 0; j < PER; j += VEC) {
                    const int e = expert_of<VEC, G>(j, lane);   // (past E within the buffer, and zero)
                    if constexpr (VEC == 4) {
                        const float4 v = *reinterpret_cast<const float4 *>(add + e);
                        d[j] += v.x;
                        d[j + 1] += v.y;
                        d[j + 2] += v.z;
                        d[j + 3] += v.w;
                    } else {
                        d[j] += add[e];
                    }
                }
                __syncwarp();
                if (on) add[id] = 0.0f;
                __syncwarp();
            }
        }
        if (R > 1) {   // rows that have no gradient, beside others that do
            if (t >= end) continue;
            if (!inside)
#pragma unroll
                for (int j = 0; j < PER; ++j) d[j] = 0.0f;
        }
        D *row = static_cast<D *>(p.dlogits) + (size_t)t * p.E;
        if constexpr (VEC == 4) {
#pragma unroll
            for (int j = 0; j < PER; j += 4) {
                const int e = expert_of<4, G>(j, lane);
                if (e >= p.E) continue;
                union {
                    uint4 q;
                    uint2 h;
                    D d[4];
                } u;
                pair_from_f32(u.d, d[j], d[j + 1]);
                pair_from_f32(u.d + 2, d[j + 2], d[j + 3]);
                if constexpr (sizeof(D) == 4) *reinterpret_cast<uint4 *>(row + e) = u.q;
                else *reinterpret_cast<uint2 *>(row + e) = u.h;
            }
        } else {
#pragma unroll
            for (int j = 0; j < PER; ++j) {
                const int e = expert_of<1, G>(j, lane);
                if (e < p.E) from_f32(row[e], d[j]);
            }
        }
    }
}

// tokens of a CTA where `ctas` of them are wanted
int chunk_tokens(int T, int ctas = kMaxChunks)
{
    return std::max(kMinChunk, ((T + ctas - 1) / ctas + kWarps - 1) / kWarps * kWarps);
}

struct BalanceLayout {
    size_t psum, pcount, pmeta, ploss, total;
};

BalanceLayout balance_layout(int T, int E, int S)
{
    const auto up = [](size_t v) { return (v + 255) / 256 * 256; };
    const size_t slots = (size_t)std::min(kMaxChunks, (T + kMinChunk - 1) / kMinChunk) + S;   // of T tokens or fewer
    BalanceLayout L;
    L.psum = 256;
    L.pcount = L.psum + up(slots * E * 4);
    L.pmeta = L.pcount + up(slots * E * 4);
    L.ploss = L.pmeta + up(slots * 8);
    L.total = L.ploss + up((size_t)S * ((E + 31) / 32) * 4);
    return L;
}

// f(logits that a lane holds, VEC, lanes) for rows of E; K places fit the lanes too.  What a row costs beside its logits (the
// sums over its lanes, the places' gradients) is shared by the rows that a warp takes at once, until the registers
// leave too few warps.  Microseconds of 65536 tokens, both directions, by 32, 16 and 8 lanes a row: 30 experts 44, 34, 24;
// 64 48, 33, 26; 128 50, 34, 33 (8192 tokens 16.9, 16.4, 17.6); 192 54, 42; 256 59, 51, of which forward 20.7, 21.9;
// 384 73.4, 73.6.
template <bool GRAD, typename F>
cudaError_t with_row(int E, int K, bool four, F &&f)
{
    const auto go = [&](auto per, auto lanes) {
        return four ? f(per, std::integral_constant<int, 4>(), lanes) : f(per, std::integral_constant<int, 1>(), lanes);
    };
#define ROW(per, lanes) go(std::integral_constant<int, per>(), std::integral_constant<int, lanes>())
    if (E <= 32 && K <= 8) return ROW(4, 8);
    if (E <= 64 && K <= 8) return ROW(8, 8);
    if (E <= 128) return ROW(8, 16);
    if (E <= 192) return ROW(12, 16);
    if (E <= 256) return ROW(GRAD ? 16 : 8, GRAD ? 16 : 32);
    if (E <= 384) return ROW(12, 32);
    return ROW(16, 32);
#undef ROW
}

int elem_bytes(int dtype) { return dtype == MOE_DTYPE_F32 ? 4 : 2; }

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

// four logits at a time where every row allows it
bool by_four(const BalanceArgs &a, int dtype) { return a.E % 4 == 0 && a.ld % 4 == 0 && !off(a.logits, 4 * elem_bytes(dtype)); }

// One kernel where the last CTA has few sums (of a chunk and expert) to add, else a second one.  Microseconds, one
// kernel and two: 16 tokens of 64 experts (128 sums) 5.5, 7.3; 64 of 64 in 3 sequences (448) 8.4, 9.3; 64 of 256
// (1280) 8.7, 7.6; 256 of 256 (4352) 18.0, 7.6.
constexpr int kFinishSums = 1024;

cudaError_t launch_forward(BalanceArgs a, int dtype, cudaStream_t st)
{
    const long long chunks = (a.T + a.chunk - 1) / a.chunk;
    a.finish = a.T > 0 && (chunks + a.S) * a.E <= kFinishSums;
    if (a.T > 0) {
        const cudaError_t e = with_dtype(dtype, [&](auto t) {
            return with_row<false>(a.E, a.K, by_four(a, dtype), [&](auto per, auto vec, auto lanes) {
                return launch_kernel(balance_parts_kernel<decltype(t), decltype(per)::value, decltype(vec)::value, decltype(lanes)::value>,
                                     dim3((unsigned)chunks), dim3(32 * kWarps), 0, st, 1, a);
            });
        });
        if (e != cudaSuccess || a.finish) return e;
    }
    // a warp for each slot of a sequence in the mean, four at least: 2000 sequences of ten tokens take 34 us, with one
    // warp 64 and with sixteen 54
    const int warps = (int)std::min<long long>(kLossWarps, std::max<long long>(4, (chunks + a.S - 1) / a.S));
    return launch_kernel(balance_loss_kernel, dim3(a.S, (a.E + 31) / 32), dim3(32 * warps), 0, st, 1, a);
}

cudaError_t launch_backward(const BalanceArgs &a, int dtype, int gdtype, cudaStream_t st)
{
    const bool four = by_four(a, dtype) && !off(a.dlogits, 4 * elem_bytes(gdtype));
    return with_dtype(dtype, [&](auto t) {
        return with_row<true>(a.E, a.K, four, [&](auto per, auto vec, auto lanes) {
            using T = decltype(t);
            constexpr int PER = decltype(per)::value, VEC = decltype(vec)::value, G = decltype(lanes)::value;
            BalanceArgs b = a;
            b.chunk = chunk_tokens(a.T, 152 * grad_ctas(PER));
            const dim3 grid((a.T + b.chunk - 1) / b.chunk);
            return gdtype == dtype ? launch_kernel(balance_backward_kernel<T, T, PER, VEC, G>, grid, dim3(32 * kWarps), 0, st, 1, b)
                                   : launch_kernel(balance_backward_kernel<T, float, PER, VEC, G>, grid, dim3(32 * kWarps), 0, st, 1, b);
        });
    });
}

#define BALANCE_PTR(p, a)                                                                               \
    do {                                                                                                \
        if (!(p)) return set_error(MOE_ERR_ARG, "%s is NULL", #p);                                      \
        if (off((p), (a))) return set_error(MOE_ERR_ALIGN, "%s is not %d-byte aligned", #p, (int)(a));  \
    } while (0)

int check_balance(const moe_config *cfg, const void *logits, int dtype, long long ld, const int32_t *ids, const int32_t *keff, int T,
                  const int32_t *offsets, int S, const int32_t *counts, const int32_t *tokens)
{
    int rc;
    if ((rc = validate_config(cfg, T))) return rc;
    if (dtype != MOE_DTYPE_F32 && dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16)
        return set_error(MOE_ERR_ARG, "unknown dtype %d", dtype);
    if (ld < cfg->n_experts) return set_error(MOE_ERR_SHAPE, "ld must be at least n_experts (got %lld)", ld);
    if (S < 1 || S > kMaxSequences) return set_error(MOE_ERR_SHAPE, "n_seq must be in [1, 2^20] (got %d)", S);
    BALANCE_PTR(offsets, 4);
    BALANCE_PTR(counts, 4);
    BALANCE_PTR(tokens, 4);
    if (T == 0) return MOE_OK;
    BALANCE_PTR(logits, elem_bytes(dtype));
    BALANCE_PTR(ids, 4);
    BALANCE_PTR(keff, 4);
    return MOE_OK;
}

int check_workspace(void *ws, size_t bytes, size_t need)
{
    if (!ws) return set_error(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (off(ws, 256)) return set_error(MOE_ERR_ALIGN, "workspace is not 256-byte aligned");
    if (bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace has %zu bytes; %zu needed", bytes, need);
    return MOE_OK;
}

int done(cudaError_t e, const char *what)
{
    if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return set_error(MOE_OK, "%s", "");
}

BalanceArgs arguments(const moe_config *cfg, const void *logits, long long ld, const int32_t *ids, const int32_t *keff, int T,
                      const int32_t *offsets, int S, const uint8_t *valid, const int32_t *counts, const int32_t *tokens, void *ws)
{
    BalanceArgs a = {};
    a.logits = logits;
    a.ld = ld;
    a.ids = ids;
    a.keff = keff;
    a.offsets = offsets;
    a.valid = valid;
    a.T = T;
    a.E = cfg->n_experts;
    a.K = cfg->top_k;
    a.S = S;
    a.chunk = chunk_tokens(T);
    a.counts = const_cast<int32_t *>(counts);
    a.tokens = const_cast<int32_t *>(tokens);
    a.scale = cfg->routed_scaling_factor;
    a.norm = cfg->norm_topk_prob;
    a.err = static_cast<int32_t *>(ws);
    a.ticket = a.err + 1;
    return a;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" {

size_t moe_balance_workspace_size(const moe_config *cfg, int max_tokens, int max_seq)
{
    if (validate_config(cfg, max_tokens) || max_seq < 1 || max_seq > kMaxSequences) return 0;
    return balance_layout(max_tokens, cfg->n_experts, max_seq).total;
}

int moe_balance_forward(const moe_config *cfg, const void *logits, int dtype, long long ld, const int32_t *ids, const int32_t *keff,
                        int T, const int32_t *seq_offsets, int n_seq, const uint8_t *valid, float *loss, int32_t *counts,
                        int32_t *tokens, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_balance(cfg, logits, dtype, ld, ids, keff, T, seq_offsets, n_seq, counts, tokens))) return rc;
    BALANCE_PTR(loss, 4);
    const BalanceLayout L = balance_layout(T, cfg->n_experts, n_seq);
    if ((rc = check_workspace(workspace, workspace_bytes, L.total)) || (rc = require_device())) return rc;
    BalanceArgs a = arguments(cfg, logits, ld, ids, keff, T, seq_offsets, n_seq, valid, counts, tokens, workspace);
    char *ws = static_cast<char *>(workspace);
    a.psum = reinterpret_cast<float *>(ws + L.psum);
    a.pcount = reinterpret_cast<int32_t *>(ws + L.pcount);
    a.pmeta = reinterpret_cast<int32_t *>(ws + L.pmeta);
    a.ploss = reinterpret_cast<float *>(ws + L.ploss);
    a.loss = loss;
    return done(launch_forward(a, dtype, (cudaStream_t)stream), "balance loss launch");
}

int moe_balance_backward(const moe_config *cfg, const void *logits, int dtype, long long ld, const int32_t *ids, const int32_t *keff,
                         int T, const int32_t *seq_offsets, int n_seq, const uint8_t *valid, const int32_t *counts,
                         const int32_t *tokens, const float *dloss, const float *dw, void *dlogits, int grad_dtype, void *workspace,
                         size_t workspace_bytes, void *stream)
{
    int rc;
    if ((rc = check_balance(cfg, logits, dtype, ld, ids, keff, T, seq_offsets, n_seq, counts, tokens))) return rc;
    if (grad_dtype != dtype && grad_dtype != MOE_DTYPE_F32)
        return set_error(MOE_ERR_ARG, "grad_dtype must be dtype or fp32 (got %d)", grad_dtype);
    if (!dloss && !dw) return set_error(MOE_ERR_ARG, "dloss and dw are both NULL");
    if (off(dloss, 4) || off(dw, 4)) return set_error(MOE_ERR_ALIGN, "dloss or dw is not 4-byte aligned");
    if (T == 0) return done(cudaSuccess, "");
    BALANCE_PTR(dlogits, elem_bytes(grad_dtype));
    if ((rc = check_workspace(workspace, workspace_bytes, 256)) || (rc = require_device())) return rc;
    BalanceArgs a = arguments(cfg, logits, ld, ids, keff, T, seq_offsets, n_seq, valid, counts, tokens, workspace);
    a.dloss = dloss;
    a.dw = dw;
    a.dlogits = dlogits;
    return done(launch_backward(a, dtype, grad_dtype, (cudaStream_t)stream), "balance gradient launch");
}

}  // extern "C"
