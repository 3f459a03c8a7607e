// gemm16.cuh -- the 16-bit matrix products of the gated block on pairs of SMs (tcgen05
// cta_group::2): output rows on the accumulator's lanes, output columns on its columns.
//   kGate2   h = silu(x Wg^T) * (x Wu^T)     rows T, columns F; two column operands, two sums
//   kDx      dx = dg Wg + du Wu              rows T, columns H; two phases of the reduction
//   kDw      dWg = dg^T x, dWu = du^T x      rows F, columns H; two groups of tiles
//
// Why pairs: a 128 x 256 tile of one SM moves 48 KB into shared memory and 48 KB out of it for
// 512 cycles of the tensor pipe, 192 bytes a cycle where shared memory gives 128 and L2 about 64
// into an SM; that form stood at 1.28 PFLOP/s.  A pair works on 256 x 256, each SM holding its
// 128 rows and half of the columns' operand: 32 KB in and out.
//
// A thread of the epilogue holds consecutive columns of one output row, so that it writes 32
// bytes at a time with no exchange between lanes.
//
// Tiles: 256 rows x `width` columns (a multiple of 32, chosen by the host so that the tiles
// fill whole waves of SM pairs).  Warps of each CTA: 0-7 its operand loads, one TMA box
// of every second stage each (a box costs the warp that issues it about 270 cycles beside its 1.8
// a row, and boxes of different warps overlap: three boxes of a stage from one warp held the stage
// at 700 cycles), then the epilogue, two or four for each quarter of the lanes, then one that issues
// the leader's MMAs.
// Barriers: `full` lives in
// the leader (both CTAs' copies complete on it); `empty` and `dfull` are in both (multicast
// commits); `dempty` in the leader (both epilogues arrive).  Waits are bounded as in gemm_tc.cuh.
#pragma once

#include "gemm_tc.cuh"

namespace moe {
namespace gemm16 {

using gemm::commit_pair;
using gemm::expect_tx;
using gemm::tma_2d_pair;
using gemm::uniform;

enum Mode { kGate2, kDx, kDw };

constexpr int kLanes = 128;   // rows of a CTA (a pair: 256)
constexpr int kMaxCols = 256;
constexpr int kBoxes = 4;                     // TMA boxes of a stage, at most
constexpr int kWarpEpi = 2 * kBoxes;

constexpr bool rows_mn(Mode m) { return m == kDw; }    // rows operand stored reduction-major
constexpr bool cols_mn(Mode m) { return m != kGate2; }

struct Args {
    int rows, cols;          // of the output (one group)
    int mtiles, ntiles;      // 256-row tiles, column chunks
    int width;               // columns of a chunk, a multiple of 32, at most 256
    int groups;              // kDw: 2 (gate, up)
    int rbox;                // rows of the rows operand's box: 128, or what a call of fewer has (the
                             // lanes after them hold whatever was there; none of them is stored)
    int ksteps, kphase;      // stages of 64; kDx: stages of the first phase
    void *out[3];            // (h, kept dh/dg, dh/du) | dx | (dWg, dWu)
    int stages, stage_bytes; // of the ring: a tile of few rows and columns has more and smaller ones
    int rows_bytes;          // the rows operand's part of a stage
    int cols_bytes;          // one columns operand's
    int dtype;
    int wide;                // rows and outputs lie on 32-byte boundaries
    uint32_t idesc;          // without N
    int32_t *err;
};

struct Maps {
    CUtensorMap r[2];   // rows operand, by phase (kDx) or group (kDw): boxes of 128 rows, or 64 x 64
    CUtensorMap c[2];   // columns operand: gate, up (kGate2) or by phase: boxes of width / 2 rows, or 64 x 64
};

template <Mode MODE>
struct Cfg {
    static constexpr int NB = MODE == kGate2 ? 2 : 1;
    static constexpr int NBUF = MODE == kGate2 ? 1 : 2;
    // Epilogue warps, and columns that one reads at a time.  The gate's two sums fill TMEM, so no MMA
    // runs beside its epilogue: twice the warps on half the columns each (4096 x 6144 x 2048 with
    // what it kept then 122.6 us, with eight warps 128.4; with what it keeps now 124).
    static constexpr int EPI = MODE == kGate2 ? 16 : 8;
    static constexpr int READ = MODE == kGate2 ? 16 : 32;
    static constexpr int MMA_WARP = kWarpEpi + EPI;
    static constexpr int THREADS = 32 * (MMA_WARP + 1);
};

constexpr int kMaxStages = 16;
constexpr int kRingBytes = 13 * 16384;   // the MMA reads 16 KB from a stage's rows, however few they are
constexpr int kSmemBytes = 1024 + kRingBytes + 512;

struct Ctrl {
    uint64_t full[kMaxStages], empty[kMaxStages], dfull[2], dempty[2], fin;
    uint32_t tmem;
    int abort;
};

// descriptor of an operand tile stored reduction-major (64 lanes or columns of 128 bytes per
// reduction index, 128-byte swizzle): 64-wide chunks 8192 bytes apart, 8 reduction indices 1024
__device__ __forceinline__ uint64_t sdesc_mn_sw128(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(8192u >> 4) << 16 | (uint64_t)(1024u >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

__device__ __forceinline__ bool stopped(const Ctrl *c) { return aborted(&c->abort); }

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Ctrl *c, int32_t *err)
{
    return wait_or_abort(bar, parity, &c->abort, err);
}

__device__ __forceinline__ void mma_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&v)[16]) { tc::ld16(taddr, v); }
__device__ __forceinline__ void ld_cols(uint32_t taddr, uint32_t (&v)[32]) { tc::ld32(taddr, v); }

// two consecutive columns
__device__ __forceinline__ uint32_t pack2(float lo, float hi, int dtype)
{
    if (dtype == MOE_DTYPE_BF16) {
        const __nv_bfloat162 p = __floats2bfloat162_rn(lo, hi);
        return *reinterpret_cast<const uint32_t *>(&p);
    }
    const __half2 p = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t *>(&p);
}

// 16 columns of a row (32 bytes), those below `n`: one 32-byte store where rows allow it (a whole
// sector a lane: 16-byte stores of 32 rows each are as many requests), else 16 bytes at a time
__device__ __forceinline__ void put32(void *out, size_t at, const uint32_t (&w)[8], int n, const Args &a)
{
    char *p = static_cast<char *>(out) + at * 2;
    if (a.wide && n >= 16) {
        asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
                     "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                     : "memory");
    } else {
        *reinterpret_cast<uint4 *>(p) = make_uint4(w[0], w[1], w[2], w[3]);
        if (n >= 16) *reinterpret_cast<uint4 *>(p + 16) = make_uint4(w[4], w[5], w[6], w[7]);
    }
}

// h, and the kept factors where they are asked for, of 16 columns
template <bool FP16>
__device__ __forceinline__ void put_gated(const float (&g)[16], const float (&u)[16], size_t at, int n, const Args &a)
{
    uint32_t h[8];
    if (!a.out[1]) {
#pragma unroll
        for (int i = 0; i < 8; ++i) h[i] = pack2(gemm::silu(g[2 * i]) * u[2 * i], gemm::silu(g[2 * i + 1]) * u[2 * i + 1], a.dtype);
        put32(a.out[0], at, h, n, a);
        return;
    }
    uint32_t ka[8], kb[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        float A[2], B[2];
        const float h0 = gated(g[2 * i], u[2 * i], A[0], B[0]), h1 = gated(g[2 * i + 1], u[2 * i + 1], A[1], B[1]);
        h[i] = pack2(h0, h1, a.dtype);
        ka[i] = Kept<FP16>::code(A[0]) | Kept<FP16>::code(A[1]) << 16;
        kb[i] = Kept<FP16>::code(B[0]) | Kept<FP16>::code(B[1]) << 16;
    }
    put32(a.out[0], at, h, n, a);
    put32(a.out[1], at, ka, n, a);
    put32(a.out[2], at, kb, n, a);
}

template <Mode MODE>
__global__ void __launch_bounds__(Cfg<MODE>::THREADS, 1) gemm16_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps)
{
    using C = Cfg<MODE>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    Ctrl *c = reinterpret_cast<Ctrl *>(ring + kRingBytes);
    static_assert(sizeof(Ctrl) <= 512, "control block");
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int rank = blockIdx.x & 1, pair = blockIdx.x >> 1, pairs = gridDim.x >> 1;
    if (tid < 32) {
        if (tid < kMaxStages) {
            mbar_init(&c->full[tid], 1);
            mbar_init(&c->empty[tid], 1);
        } else if (tid < kMaxStages + 2) {
            mbar_init(&c->dfull[tid - kMaxStages], 1);
            mbar_init(&c->dempty[tid - kMaxStages], 2 * C::EPI);
        } else if (tid == 31) {
            mbar_init(&c->fin, 1);
            c->abort = 0;
        }
        fence_mbar_init();
        __syncwarp();
    }
    cluster_sync();   // both CTAs run and their barriers are ready
    if (warp == C::MMA_WARP) gemm::tmem_alloc<true>(&c->tmem, 512);
    tc::fence_before_sync();
    __syncthreads();   // (a stage is full only with the peer's copies, which follow its own allocation)
    tc::fence_after_sync();
    pdl_wait();
    pdl_launch_dependents();
    const uint32_t tmem = uniform(c->tmem);
    const int per_group = a.mtiles * a.ntiles, total = a.groups * per_group;

    if (warp < kWarpEpi) {
        // ---------------- operands by TMA: box `b` of every second stage ---------------------
        // reduction-major operands take two boxes of 64 (the second only where it is needed),
        // the others one; rows first
        constexpr int RB = rows_mn(MODE) ? 2 : 1;
        const uint32_t r0 = smem_u32(ring);
        const int b = warp % kBoxes;
        const uint32_t turn = warp / kBoxes;
        const bool of_rows = b < RB;
        const int i = of_rows ? b : b - RB;
        const int half = a.width >> 1, boxes = cols_mn(MODE) ? (half + 63) >> 6 : C::NB;
        const uint32_t bytes = 2u * ((rows_mn(MODE) ? 16384u : a.rbox * 128u) + boxes * (cols_mn(MODE) ? 8192u : half * 128u));
        const uint32_t to = r0 + (of_rows ? i * 8192 : a.rows_bytes + i * (cols_mn(MODE) ? 8192 : a.cols_bytes));
        uint32_t it = 0, s = 0, phase = 0;   // stage, and the ring's turn
        bool ok = true;
        if (of_rows || i < boxes)
            for (int t = pair; t < total && ok && !stopped(c); t += pairs) {
                const int g = t / per_group, mi = (t - g * per_group) / a.ntiles, ni = t - g * per_group - mi * a.ntiles;
                const int m0 = mi * 2 * kLanes + rank * kLanes + (rows_mn(MODE) ? 64 * i : 0);
                const int n0 = ni * a.width + rank * half + (cols_mn(MODE) ? 64 * i : 0);
                for (int ks = 0; ks < a.ksteps; ++ks, ++it, s = s + 1 == a.stages ? 0 : s + 1, phase ^= s == 0) {
                    if ((it & 1) != turn) continue;
                    if (it >= a.stages && !(ok = wait_warp(&c->empty[s], phase ^ 1, c, a.err))) break;
                    if (b == 0 && rank == 0) expect_tx(smem_u32(&c->full[s]), bytes);
                    const uint32_t bar = map_rank(smem_u32(&c->full[s]), 0);
                    const int ph = MODE == kDx && ks >= a.kphase;
                    const int k = 64 * (ph ? ks - a.kphase : ks);
                    const CUtensorMap *map = of_rows ? &maps.r[MODE == kDw ? g : ph] : &maps.c[MODE == kGate2 ? i : ph];
                    const int o = of_rows ? m0 : n0;
                    const bool mn = of_rows ? rows_mn(MODE) : cols_mn(MODE);
                    tma_2d_pair(to + s * a.stage_bytes, map, mn ? o : k, mn ? k : o, bar);
                }
            }
        if (b == 0) {
            // the leader's commits on the last stages' `empty`, which no load waits for, land before
            // this CTA ends and its shared memory is another kernel's (each warp waits for its own
            // stages: it has seen the phase before)
            for (uint32_t j = it > (uint32_t)a.stages ? it - a.stages : 0; j < it && ok; ++j)
                if ((j & 1) == turn) ok = wait_warp(&c->empty[j % a.stages], (j / a.stages) & 1, c, a.err);
        }
        __syncwarp();
    } else if (warp == C::MMA_WARP && rank == 0) {
        // ---------------- MMA issue, for both CTAs ------------------------------------------
        const uint32_t r0 = smem_u32(ring);
        uint32_t s = 0, phase = 0, nt = 0;
        bool ok = true;
        for (int t = pair; t < total && ok && !stopped(c); t += pairs, ++nt) {
            const uint32_t idesc = a.idesc | (uint32_t)(a.width >> 3) << 17;
            const uint32_t buf = nt % C::NBUF, use = nt / C::NBUF;
            if (use >= 1 && !(ok = wait_warp(&c->dempty[buf], (use - 1) & 1, c, a.err))) break;
            for (int ks = 0; ks < a.ksteps; ++ks, s = s + 1 == a.stages ? 0 : s + 1, phase ^= s == 0) {
                if (!(ok = wait_warp(&c->full[s], phase, c, a.err))) break;
                tc::fence_after_sync();
                const uint32_t rs = r0 + s * a.stage_bytes, cs = rs + a.rows_bytes;
                const uint64_t rd = rows_mn(MODE) ? sdesc_mn_sw128(rs) : tc::sdesc_kmajor_sw128(rs);
#pragma unroll
                for (int k = 0; k < 4; ++k)
#pragma unroll
                    for (int o = 0; o < C::NB; ++o) {
                        const uint64_t cd = cols_mn(MODE) ? sdesc_mn_sw128(cs) : tc::sdesc_kmajor_sw128(cs + o * a.cols_bytes);
                        mma_pair(tmem + buf * kMaxCols + o * kMaxCols, rd + (rows_mn(MODE) ? k * 128 : k * 2),
                                 cd + (cols_mn(MODE) ? k * 128 : k * 2), idesc, ks > 0 || k > 0);
                    }
                commit_pair(&c->empty[s]);
            }
            commit_pair(&c->dfull[buf]);
        }
        commit_pair(&c->fin);   // every MMA is done before TMEM is freed
    } else if (warp >= kWarpEpi && warp < C::MMA_WARP) {
        // ---------------- epilogue ----------------------------------------------------------
        const int qd = warp & 3, part = (warp - kWarpEpi) >> 2;
        const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
        uint32_t nt = 0;
        bool ok = true;
        for (int t = pair; t < total && ok && !stopped(c); t += pairs, ++nt) {
            const int g = t / per_group, mi = (t - g * per_group) / a.ntiles, ni = t - g * per_group - mi * a.ntiles;
            const int row = mi * 2 * kLanes + rank * kLanes + qd * 32 + lane, n0 = ni * a.width;
            const int n = min(a.width, a.cols - n0);
            const uint32_t buf = nt % C::NBUF, use = nt / C::NBUF;
            if (!(ok = wait_warp(&c->dfull[buf], use & 1, c, a.err))) break;
            tc::fence_after_sync();
            const size_t at = (size_t)row * a.cols + n0;
            void *out = MODE == kDw ? a.out[g] : a.out[0];
            const auto give_back = [&] {   // the accumulator, once this warp has read its part
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) gemm::arrive_cluster_relaxed(map_rank(smem_u32(&c->dempty[buf]), 0));
            };
            if (part * C::READ >= n) give_back();
            // READ columns at a time, in turns of the warps of these lanes; the width is a
            // multiple of 32, the columns of 8
            for (int c0 = part * C::READ; c0 < n; c0 += C::EPI / 4 * C::READ) {
                __syncwarp();   // lanes past the last row come from another branch, the loads want the whole warp
                uint32_t v[2][C::READ];
#pragma unroll
                for (int o = 0; o < C::NB; ++o) ld_cols(tl + buf * kMaxCols + o * kMaxCols + c0, v[o]);
                tc::wait_ld();
#pragma unroll
                for (int o = 0; o < C::NB; ++o)
#pragma unroll
                    for (int j = 0; j < C::READ; ++j) asm volatile("" : "+r"(v[o][j]));   // read after the wait
                if (c0 + C::EPI / 4 * C::READ >= n) give_back();
                if (row < a.rows) {
#pragma unroll
                    for (int j = 0; j < C::READ; j += 16) {
                        if (c0 + j >= n) break;
                        const int left = n - c0 - j;   // 8, or 16 and more
                        float x[16];
#pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = __uint_as_float(v[0][j + i]);
                        if constexpr (MODE == kGate2) {
                            float y[16];
#pragma unroll
                            for (int i = 0; i < 16; ++i) y[i] = __uint_as_float(v[1][j + i]);
                            if (a.dtype == MOE_DTYPE_F16) put_gated<true>(x, y, at + c0 + j, left, a);
                            else put_gated<false>(x, y, at + c0 + j, left, a);
                        } else {
                            uint32_t w[8];
#pragma unroll
                            for (int i = 0; i < 8; ++i) w[i] = pack2(x[2 * i], x[2 * i + 1], a.dtype);
                            put32(out, at + c0 + j, w, left, a);
                        }
                    }
                }
            }
        }
    }

    tc::fence_before_sync();
    __syncthreads();
    if (warp == C::MMA_WARP) settle(&c->fin, &c->abort);   // the leader's last commit, in both CTAs
    cluster_sync();   // neither CTA frees its TMEM or leaves while the other still uses the pair's
    if (warp == C::MMA_WARP) {
        tc::fence_after_sync();
        gemm::tmem_dealloc<true>(tmem, 512);
        __syncwarp();
    }
    cluster_sync();
}

// Column chunks: the width whose waves of SM pairs take least, by what a tile costs in cycles:
// its reduction at the tensor pipe's rate or at the 50 bytes a cycle that reach an SM from L2,
// whichever is more, and a fixed start and end.
template <Mode MODE>
void plan(Args &a)
{
    constexpr int NB = Cfg<MODE>::NB;
    const int pairs = num_sms() / 2;
    a.mtiles = (a.rows + 2 * kLanes - 1) / (2 * kLanes);
    a.rbox = std::min(kLanes, (a.rows + 15) / 16 * 16);
    double best = 0;
    for (int w = kMaxCols; w >= 32; w -= 32) {
        const long long tiles = (long long)a.groups * a.mtiles * ((a.cols + w - 1) / w);
        const double stage = std::max(2.0 * w * NB, (16384.0 + 64.0 * w * NB) / 50);
        const double cost = (double)((tiles + pairs - 1) / pairs) * (a.ksteps * stage + 3000.0 + 4.0 * w * NB);
        if (best == 0 || cost < best) {
            best = cost;
            a.width = w;
        }
    }
    a.ntiles = (a.cols + a.width - 1) / a.width;
    const int boxes = (a.width / 2 + 63) / 64;
    a.rows_bytes = MODE == kDw ? 16384 : a.rbox * 128;
    a.cols_bytes = cols_mn(MODE) ? boxes * 8192 : a.width / 2 * 128;
    a.stage_bytes = a.rows_bytes + NB * a.cols_bytes;
    a.stages = std::min(kMaxStages, (kRingBytes - 16384) / a.stage_bytes);
}

template <Mode MODE>
cudaError_t launch(Args a, const Maps &m, cudaStream_t st)
{
    uintptr_t bits = (uintptr_t)a.cols * 2;
    for (void *p : a.out) bits |= reinterpret_cast<uintptr_t>(p);
    a.wide = bits % 32 == 0;
    const long long tiles = (long long)a.groups * a.mtiles * a.ntiles;
    const int grid = 2 * (int)std::min<long long>(tiles, num_sms() / 2);
    return launch_kernel(gemm16_kernel<MODE>, dim3(grid), dim3(Cfg<MODE>::THREADS), kSmemBytes, st, 2, a, m);
}

}  // namespace gemm16
}  // namespace moe
