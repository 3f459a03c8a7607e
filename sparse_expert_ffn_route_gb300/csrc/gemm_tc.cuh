// gemm_tc.cuh -- the tcgen05 matrix-product kernel behind the MXFP4 operators and the 16-bit
// gated block for few tokens.  One kernel template, four uses:
//   kMxGate   h = q(silu(x Wg^T) * (x Wu^T)), x and W in MXFP4, h requantised to MXFP4
//   kMxMul    y = x W^T, x and W in MXFP4
//   kMxMul2   the same on twice the weight rows a tile (two lanes operands of one matrix)
//   kGate     h = silu(x Wg^T) * (x Wu^T) in 16 bits (its factors kept on request)
//
// Orientation.  The accumulator's 128 lanes are weight rows (the output's contiguous dimension)
// and its columns tokens.  A weight tile is then always a full 128-lane operand, however few tokens there
// are, and a warp's lanes write consecutive output elements.  The MMA's column count follows the
// tile's token count in steps of 16, so one token costs 16 columns.
//
// Work.  A tile is 128 lanes (256 on a pair) x up to BN columns over the whole reduction; groups
// (experts) are cut into equal column chunks.  CTAs run tiles blockIdx, blockIdx + grid, ...
//
// Many columns (BN 224) run on pairs of SMs (cta_group::2): each holds its 128 weight rows and
// half of the tokens.  What feeds the tensor pipe is the bound, about 50 bytes a cycle from L2
// into an SM: one SM's 128 x 192 tile needs 43 KB a stage for 384 cycles of the pipe and ran at
// 826 (a 4096-token prompt of 6144 x 6144 in 73 us), a pair's 256 x 224 33 KB for 448.
//
// Few columns (BN 32): with few tiles a cluster of S CTAs shares one: each takes a slice of the reduction, sends its
// partial sums to the owner of each column through distributed shared memory, and the owner
// adds them in rank order (the sums do not depend on timing).
//
// A reduction step (stage) is 128 bytes of each operand row: 64 16-bit or 256 4-bit inputs, in
// 128-byte-swizzled tiles fed by TMA.  Rows and inputs past a tensor's end are read as zero.
//
// Warps: 0, 2 and 3 feed the stages by TMA, one box of a stage each (a box costs the warp that
// issues it about 270 cycles beside its 1.8 a row, and boxes of different warps overlap): lanes
// operands on 0 and 2, the columns on 3; 1 issues the MMAs; 4-11 (4-7 for few columns) are the
// epilogue (TMEM lanes 32 * (warp % 4) ..); those after it (MXFP4 only) bring the scales, one operand of 128 rows each: global
// rows of scale bytes -> shared memory blocks of 512 bytes (row r, block k of 4 at
// 16 * (r % 32) + 4 * (r / 32) + k) that tcgen05.cp copies to TMEM.
//
// For few columns (BN 32) two CTAs fit an SM, so that a kernel of a chain starts beside the end
// of the one before it.  With `early` set the lanes operands (weights) and their scales are
// loaded before the wait for that kernel: the caller says that they and the offsets were
// complete before it began.  No bounded wait then starts before that kernel's end: the waits of
// this file measure this kernel's own progress.
//
// Every wait is bounded: one that gives up sets the workspace's error word and ends the loops of
// every CTA of the cluster (cluster_wait.cuh); what is in flight gets its time and TMEM is freed.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include <atomic>

#include "cluster_wait.cuh"
#include "device_util.cuh"
#include "gated_kept.cuh"
#include "launch.cuh"
#include "moe_internal.cuh"
#include "mx_util.cuh"
#include "tcgen05.cuh"

namespace moe {
namespace gemm {

enum Mode { kMxGate, kMxMul, kGate, kMxMul2 };

constexpr int kM = 128;          // lanes of a tile
constexpr int kBoxMaps = 7;      // column-operand maps with boxes of 16 (k + 1) rows
constexpr int kMaxGroups = 512;
constexpr int kSplitCols = 16;   // columns of a tile that CTAs share

constexpr bool is_mx(Mode m) { return m != kGate; }
constexpr bool is_gated(Mode m) { return m == kMxGate || m == kGate; }

// the kernel's parameters (tensor maps apart)
struct Args {
    const int32_t *offsets;    // [E + 1] rows of each group (null: one group of all rows)
    int E;                     // groups
    int rows;                  // columns of the output (tokens) in all
    int M;                     // lanes dimension of one group
    int ksteps;                // stages of the whole reduction
    int split;                 // CTAs that share a tile (the cluster size)
    int width;                 // columns of a tile at most (BN; kSplitCols in a cluster)
    int early;                 // weights, their scales and offsets are older than the last kernel
    // scale bytes [rows][sf_ld] of the lanes operands (groups * M rows) and the columns operand
    const uint8_t *sfa[2], *sfb;
    int sf_ld;                 // K / 32
    long long sfa_rows;        // E * M
    void *out[3];              // y | (h, kept dh/dg, dh/du) | (codes, scales)
    int ld;                    // row stride of out, in elements (codes: of M)
    int dtype;                 // MOE_DTYPE_* of out
    uint32_t idesc;            // instruction descriptor without N and the scale ids
    int32_t *err;
};

struct Maps {
    CUtensorMap a[2];
    CUtensorMap b[kBoxMaps];   // boxes of 16 (k + 1) rows: one for each number of columns that a CTA loads
};

template <Mode MODE, int BN>
struct Cfg {
    static constexpr bool MX = is_mx(MODE), GATED = is_gated(MODE);
    static constexpr int NA = GATED || MODE == kMxMul2 ? 2 : 1;   // lanes operands (accumulators) of a tile
    static constexpr bool FEW = BN <= 32;                  // clusters may share a tile
    static constexpr bool PAIR = !FEW;                     // two SMs a tile: 256 lanes, each half of the columns' operand
    static constexpr int LANES = (MODE == kMxMul2 ? 2 : 1) * (PAIR ? 2 * kM : kM);   // of a tile
    static constexpr int STEP = PAIR ? 32 : 16;            // the MMA's column count is a multiple
    static constexpr int EPI = FEW ? 4 : NA == 2 ? 16 : 8;   // epilogue warps
    // TMEM: two halves of accumulators.  A tile takes one half, so that its epilogue runs beside
    // the next tile's MMAs; two accumulators of more than HALF / 2 columns take both.
    static constexpr int HALF = FEW ? NA * BN : 224;
    static constexpr int A_BYTES = kM * 128;
    static constexpr int B_BYTES = (PAIR ? BN / 2 : BN) * 128;
    static constexpr int SFB_UNITS = MX ? (BN + 127) / 128 : 0;
    static constexpr int SF_UNITS = MX ? NA + SFB_UNITS : 0;   // 128-row scale blocks of a stage (2 x 512 B each)
    static constexpr int SF_BYTES = SF_UNITS * 1024;
    static constexpr int RED_COLS = 24;                    // >= S * ceil(16 / S) for S <= 8
    static constexpr int RED_BYTES = FEW ? NA * RED_COLS * kM * 4 : 0;
    static constexpr int CTRL_BYTES = 5120;                // control block and the groups' prefix
    static constexpr int STAGE = NA * A_BYTES + B_BYTES + SF_BYTES;
    // Two CTAs an SM where a chain of kernels overlaps (MXFP4, few columns).  The 16-bit block is one
    // kernel: one CTA with 5 stages in place of 2 (one token, weights from DRAM: 12.0 us, two CTAs
    // with 2 stages each 15.7).
    static constexpr int PER_SM = FEW && MX ? 2 : 1;
    static constexpr int BUDGET = (PER_SM == 2 ? 115712 : 232448) - 1024 - CTRL_BYTES - RED_BYTES;
    static constexpr int STAGES = BUDGET / STAGE > 8 ? 8 : BUDGET / STAGE;
    static constexpr int SMEM = 1024 + STAGES * STAGE + RED_BYTES + CTRL_BYTES;
    static constexpr int SF_WARP = 4 + EPI;
    static constexpr int THREADS = 32 * (SF_WARP + SF_UNITS);
    static constexpr int SF_COL = 2 * HALF;                // first TMEM column of the scales: 2 buffers
    static constexpr int SF_BUF = 32;                      // columns of one buffer
    static constexpr int TMEM_COLS = FEW ? 256 : 512;
    static_assert(STAGES >= 2, "shared memory budget");
    static_assert(SF_COL + (MX ? 2 * SF_BUF : 0) <= TMEM_COLS && NA * BN <= 2 * HALF, "TMEM budget");
    static constexpr bool both_halves(int np) { return NA * np > HALF; }
};

// A value that all lanes hold alike, in a form that the compiler knows to be uniform: operands of
// the MMA and TMA instructions live in uniform registers, and moving them there from ordinary
// ones for each instruction held the issue of a stage's MMAs and copies at 50 to 70 cycles each.
__device__ __forceinline__ uint32_t uniform(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }
__device__ __forceinline__ int uniform(int v) { return __reduce_max_sync(0xffffffffu, v); }

struct Ctrl {
    uint64_t full[8], empty[8], sfull[8], dfull[2], dempty[2], rfull, rempty, fin;
    uint32_t tmem;
    int abort;
    int tiles;
    int warp_tiles[24];
    int32_t prefix[kMaxGroups + 1], off[kMaxGroups + 1];
};

__device__ __forceinline__ bool stopped(const Ctrl *c) { return aborted(&c->abort); }

__device__ __forceinline__ bool wait_warp(uint64_t *bar, uint32_t parity, Ctrl *c, int32_t *err)
{
    return wait_or_abort(bar, parity, &c->abort, err);
}

// the same on a barrier that other CTAs of the cluster arrive at (their writes become visible)
__device__ __forceinline__ bool wait_warp_cluster(uint64_t *bar, uint32_t parity, Ctrl *c, int32_t *err)
{
    return wait_or_abort<true>(bar, parity, &c->abort, err);
}

__device__ __forceinline__ void tma_2d(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void expect_tx(uint32_t bar, uint32_t bytes)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
        : "memory");
}

// descriptor of a 512-byte scale block: 32 rows of 16 bytes, no swizzle, 8-row groups 128 apart
__device__ __forceinline__ uint64_t sdesc_scales(uint32_t saddr)
{
    return (uint64_t)((saddr & 0x3FFFFu) >> 4) | (uint64_t)(128u >> 4) << 16 | (uint64_t)(128u >> 4) << 32 |
           (uint64_t)1 << 46;
}

__device__ __forceinline__ void mma_f16(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
        "l"(a), "l"(b), "r"(idesc), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void mma_mx4(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                        uint32_t sfb, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::1.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

__device__ __forceinline__ void cp_scales(uint32_t taddr, uint64_t desc)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::1.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
        "l"(desc)
        : "memory");
}

// one 32-bit column of this thread's TMEM lane from each of N accumulators, `step` columns apart
template <int N>
__device__ __forceinline__ void ld1(uint32_t taddr, uint32_t step, uint32_t (&v)[2])
{
    v[1] = 0;
    if constexpr (N == 2)
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%2];\n\t"
            "tcgen05.ld.sync.aligned.32x32b.x1.b32 {%1}, [%3];\n\t"
            "tcgen05.wait::ld.sync.aligned;"
            : "=r"(v[0]), "=r"(v[1])
            : "r"(taddr), "r"(taddr + step)
            : "memory");
    else
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];\n\ttcgen05.wait::ld.sync.aligned;"
                     : "=r"(v[0])
                     : "r"(taddr)
                     : "memory");
}

// --- cluster ----------------------------------------------------------------------------
// asynchronous 4-byte store into another CTA's shared memory that counts on a barrier there
__device__ __forceinline__ void st_async(uint32_t addr, uint32_t v, uint32_t bar)
{
    asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.b32 [%0], %1, [%2];" ::"r"(addr), "r"(v), "r"(bar)
                 : "memory");
}
__device__ __forceinline__ void arrive_cluster(uint32_t bar)
{
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
// the same for what needs no order of memory, the end of TMEM reads (a release at cluster scope waits
// for the warp's global stores, 1500 cycles and more)
__device__ __forceinline__ void arrive_cluster_relaxed(uint32_t bar)
{
    asm volatile("mbarrier.arrive.relaxed.cluster.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }

// --- pairs of SMs (cta_group::2) ---------------------------------------------------------
// TMA into this CTA's shared memory, completing on a barrier of either CTA of the pair
__device__ __forceinline__ void tma_2d_pair(uint32_t dst, const CUtensorMap *map, int x, int y, uint32_t bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 "
        "[%0], [%1, {%2, %3}], [%4];\n\t}" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}

// one arrival on this barrier of both CTAs once the tensor operations issued so far are done
__device__ __forceinline__ void commit_pair(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 3;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
}

// one arrival on this barrier of the pair's leader
__device__ __forceinline__ void commit_leader(uint64_t *bar)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\t.reg .b16 m;\n\tmov.b16 m, 1;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], m;\n\t}" ::"r"(
            smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void mma_mx4_pair(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t sfa,
                                             uint32_t sfb, uint32_t acc)
{
    asm volatile(
        "{\n\t.reg .pred p, e;\n\telect.sync _|e, 0xffffffff;\n\tsetp.ne.b32 p, %6, 0;\n\t"
        "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%0], %1, %2, %3, [%4], [%5], p;\n\t}" ::"r"(
            d),
        "l"(a), "l"(b), "r"(idesc), "r"(sfa), "r"(sfb), "r"(acc)
        : "memory");
}

// each CTA's block at this place of its shared memory into its TMEM
__device__ __forceinline__ void cp_scales_pair(uint32_t taddr, uint64_t desc)
{
    asm volatile(
        "{\n\t.reg .pred e;\n\telect.sync _|e, 0xffffffff;\n\t"
        "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t}" ::"r"(taddr),
        "l"(desc)
        : "memory");
}

template <bool PAIR>
__device__ __forceinline__ void commit(uint64_t *bar)
{
    if constexpr (PAIR) commit_pair(bar);
    else tc::commit_elect(bar);
}

// TMEM of a CTA, or of both CTAs of a pair.  The pair's forms are issued by a warp of each CTA, and
// neither may issue while the other CTA has not started or has ended: a cluster barrier of all
// threads stands before the allocation and one after the freeing.
template <bool PAIR>
__device__ __forceinline__ void tmem_alloc(uint32_t *dst, uint32_t cols)
{
    if constexpr (PAIR) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(dst)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tc::tmem_alloc(dst, cols);
        tc::tmem_relinquish();
    }
}

template <bool PAIR>
__device__ __forceinline__ void tmem_dealloc(uint32_t taddr, uint32_t cols)
{
    if constexpr (PAIR) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(cols) : "memory");
    else tc::tmem_dealloc(taddr, cols);
}

// --- tiles ------------------------------------------------------------------------------
struct Tile {
    int e, m0, row0, n, np;
};

// columns of a group of c rows in nt chunks of equal size (a multiple of 16)
__device__ __forceinline__ int chunk_cols(int c, int nt) { return ((c + nt - 1) / nt + 15) & ~15; }

template <class C>
__device__ __forceinline__ Tile get_tile(const Args &a, const Ctrl *ctrl, int t)
{
    // the last group with prefix <= t, in two looks of the warp: which 16 groups, which of them
    const int lane = threadIdx.x & 31;
    const int k = 31 - __clz(__ballot_sync(0xffffffffu, 16 * lane < a.E && ctrl->prefix[16 * lane] <= t));
    const int at = 16 * k + (lane & 15);
    const int lo = 16 * k + 31 - __clz(__ballot_sync(0xffffffffu, lane < 16 && at < a.E && ctrl->prefix[at] <= t));
    const int first = a.offsets ? uniform(ctrl->off[lo]) : 0;
    const int rows = a.offsets ? uniform(ctrl->off[lo + 1]) - first : a.rows;
    const int nt = rows > a.width ? (rows + a.width - 1) / a.width : 1;
    const int w = nt == 1 ? rows : chunk_cols(rows, nt);
    const int local = t - uniform(ctrl->prefix[lo]);
    const int mi = nt == 1 ? local : local / nt, ni = local - mi * nt;   // a weight tile's chunks run next to one another
    Tile r;
    r.e = lo;
    r.m0 = mi * C::LANES;   // the pair's first lane
    r.row0 = first + ni * w;
    r.n = max(0, min(w, rows - ni * w));
    r.np = max(C::STEP, (r.n + C::STEP - 1) & ~(C::STEP - 1));
    return r;
}

__device__ __forceinline__ float silu(float g) { return __fdividef(g, 1.0f + __expf(-g)); }

__device__ __forceinline__ void store(void *p, int dtype, size_t i, float v)
{
    if (dtype == MOE_DTYPE_F32) reinterpret_cast<float *>(p)[i] = v;
    else if (dtype == MOE_DTYPE_BF16) reinterpret_cast<__nv_bfloat16 *>(p)[i] = __float2bfloat16_rn(v);
    else reinterpret_cast<__half *>(p)[i] = __float2half_rn(v);
}

// 8 columns of h of this lane's row -> MXFP4.  A block is the warp's 32 rows of one column.
// col(j) gives column j's output row, or -1.
template <class Col>
__device__ __forceinline__ void emit_mx8(const Args &a, const float (&v)[8], int m, int lane, Col col)
{
    // (of a block with a NaN or an infinity the codes do not matter: its scale is NaN)
    uint32_t w = 0, sbs[2] = {0, 0};   // the columns' scale bytes, the same in all lanes
#pragma unroll
    for (int j = 0; j < 8; j += 2) {
        float s[2];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            float f;
            const uint32_t sb = mx_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(v[j + k]) & 0x7fffffffu), f);
            s[k] = v[j + k] * f;
            sbs[j >> 2] |= sb << (8 * ((j + k) & 3));
        }
        w |= e2m1x2(s[0], s[1]) << (4 * j);
    }
    const uint32_t mine = (lane & 4 ? sbs[1] : sbs[0]) >> (8 * (lane & 3));
    // lane 8a + i holds column j's nibble of row 8a + i at nibble j: transpose within 8 lanes,
    // so that lane 8a + j holds rows 8a .. 8a + 7 of column j
#pragma unroll
    for (int d = 4; d; d >>= 1) {
        const uint32_t mask = d == 4 ? 0x0000ffffu : d == 2 ? 0x00ff00ffu : 0x0f0f0f0fu;
        const bool up = lane & d;
        const uint32_t got = __shfl_xor_sync(0xffffffffu, up ? (w & mask) : ((w >> (4 * d)) & mask), d);
        w = up ? ((w & ~mask) | got) : ((w & mask) | (got << (4 * d)));
    }
    const int r = col(lane & 7);
    if (r >= 0 && m < a.M) {
        const size_t at = (size_t)r * a.ld + (m & ~7);   // first of the 8 rows that this word holds
        *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.out[0]) + (at >> 1)) = w;
        if (lane < 8) static_cast<uint8_t *>(a.out[1])[(size_t)r * (a.ld >> 5) + (m >> 5)] = (uint8_t)mine;
    }
}

// 16 columns of a tile -> the outputs; col(j): column j's output row, or -1
template <Mode MODE, class Col>
__device__ __forceinline__ void emit16(const Args &a, const float (&g)[16], const float (&u)[16], int m, int lane, Col col)
{
    if constexpr (MODE == kMxGate) {
#pragma unroll
        for (int j0 = 0; j0 < 16; j0 += 8) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = silu(g[j0 + j]) * u[j0 + j];
            emit_mx8(a, v, m, lane, [&](int j) { return col(j0 + j); });
        }
    } else {
#pragma unroll
        for (int o = 0; o < (MODE == kMxMul2 ? 2 : 1); ++o) {
            const int n = m + 2 * kM * o;
            if (n >= a.M) return;
#pragma unroll
            for (int j = 0; j < 16; ++j) {
                const int r = col(j);
                if (r >= 0) store(a.out[0], a.dtype, (size_t)r * a.ld + n, o ? u[j] : g[j]);
            }
        }
    }
}

// One column of a tile (few columns): row `r` of the output.  A rolled loop over the columns in
// place of the unrolled 16 keeps the code of a one-token call small: there every instruction is
// fetched once and used once.
template <Mode MODE>
__device__ __forceinline__ void emit1(const Args &a, float g, float u, int m, int lane, int r)
{
    if constexpr (MODE == kMxGate) {
        const float v = silu(g) * u;
        float f;
        const uint32_t sb = mx_scale(__reduce_max_sync(0xffffffffu, __float_as_uint(v) & 0x7fffffffu), f);
        uint32_t w = e2m1x2(f == 0.0f ? 0.0f : v * f, 0.0f) << (4 * (lane & 7));
#pragma unroll
        for (int d = 1; d < 8; d <<= 1) w |= __shfl_xor_sync(0xffffffffu, w, d);
        if (m < a.M) {
            const size_t at = (size_t)r * a.ld + m;
            if ((lane & 7) == 0) *reinterpret_cast<uint32_t *>(static_cast<uint8_t *>(a.out[0]) + (at >> 1)) = w;
            if (lane == 0) static_cast<uint8_t *>(a.out[1])[at >> 5] = (uint8_t)sb;
        }
    } else if (m < a.M) {
        const size_t at = (size_t)r * a.ld + m;
        if constexpr (MODE == kGate) {
            float A, B;
            store(a.out[0], a.dtype, at, gated(g, u, A, B));
            if (a.out[1]) {
                const bool f16 = a.dtype == MOE_DTYPE_F16;
                static_cast<uint16_t *>(a.out[1])[at] = (uint16_t)(f16 ? Kept<true>::code(A) : Kept<false>::code(A));
                static_cast<uint16_t *>(a.out[2])[at] = (uint16_t)(f16 ? Kept<true>::code(B) : Kept<false>::code(B));
            }
        } else {
            store(a.out[0], a.dtype, at, g);
        }
    }
}

// 16 scale bytes (blocks 16 kc .. 16 kc + 15) of a row of K / 32; past the end: 0 (2^-127, on
// codes that are zero there).  load() only starts the loads, get() uses them, so that a chunk's
// loads run beside the stores of the one before.
template <bool WHOLE>
struct Scales;

// K is a multiple of 512: every row's 16 bytes are one aligned load.  A kernel of its own, since the
// other form's code beside it cost one-token calls a microsecond.
template <>
struct Scales<true> {
    uint4 v;
    __device__ __forceinline__ void load(const uint8_t *base, long long row, long long rows, int ld, int kc)
    {
        v = make_uint4(0, 0, 0, 0);
        if (row < rows) v = __ldg(reinterpret_cast<const uint4 *>(base + row * ld + 16 * kc));
    }
    __device__ __forceinline__ uint4 get() const { return v; }
};

// Otherwise the two aligned 16 bytes around them, shifted into place (2000 x 4000 x 2528 in 20 us;
// byte loads 35).  The last row's may pass the array's end by up to 15 bytes, never a 16-byte
// boundary: the entry points ask for arrays that are readable up to the next one.
template <>
struct Scales<false> {
    uint4 lo, hi;
    int sh, left;   // bytes before them in lo, bytes of the row from here on
    __device__ __forceinline__ void load(const uint8_t *base, long long row, long long rows, int ld, int kc)
    {
        const long long o = row * ld + 16 * kc;
        sh = (int)o & 15;
        left = row < rows ? ld - 16 * kc : 0;
        lo = hi = make_uint4(0, 0, 0, 0);
        const uint4 *p = reinterpret_cast<const uint4 *>(base + (o - sh));
        if (left > 0) lo = __ldg(p);
        if (sh + min(left, 16) > 16) hi = __ldg(p + 1);
    }
    __device__ __forceinline__ uint4 get() const
    {
        const uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
        uint32_t x[6], y[5], r[4];
#pragma unroll
        for (int i = 0; i < 6; ++i) x[i] = sh & 8 ? w[i + 2] : w[i];
#pragma unroll
        for (int i = 0; i < 5; ++i) y[i] = sh & 4 ? x[i + 1] : x[i];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[i] = __funnelshift_r(y[i], y[i + 1], 8 * (sh & 3));
            const int keep = left - 4 * i;   // valid bytes of this word
            if (keep < 4) r[i] &= keep > 0 ? (1u << (8 * keep)) - 1u : 0u;
        }
        return make_uint4(r[0], r[1], r[2], r[3]);
    }
};

template <Mode MODE, int BN, bool WHOLE>
__global__ void __launch_bounds__(Cfg<MODE, BN>::THREADS, Cfg<MODE, BN>::PER_SM)
    gemm_kernel(const __grid_constant__ Args a, const __grid_constant__ Maps maps)
{
    using C = Cfg<MODE, BN>;
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *sfring = ring + C::STAGES * (C::NA * C::A_BYTES + C::B_BYTES);
    float *red = reinterpret_cast<float *>(sfring + C::STAGES * C::SF_BYTES);
    Ctrl *c = reinterpret_cast<Ctrl *>(reinterpret_cast<uint8_t *>(red) + C::RED_BYTES);
    static_assert(sizeof(Ctrl) <= C::CTRL_BYTES, "control block");
    const int tid = threadIdx.x, warp = uniform(tid >> 5), lane = tid & 31;
    const int mtiles = (a.M + C::LANES - 1) / C::LANES;
    const int S = C::FEW ? a.split : 1;
    // CTAs of a cluster: S that share a tile's reduction, or the two of a pair
    const int CS = C::PAIR ? 2 : S;
    const int rank = (int)(blockIdx.x % CS), tile0 = (int)(blockIdx.x / CS), tstep = (int)(gridDim.x / CS);
    const int ks0 = C::PAIR ? 0 : (int)((long long)a.ksteps * rank / S);
    const int ks1 = C::PAIR ? a.ksteps : (int)((long long)a.ksteps * (rank + 1) / S);
    const int lane0 = C::PAIR ? rank * kM : 0;   // this CTA's first lane in the tile

    if (tid < 32) {
        if (tid < C::STAGES) {
            mbar_init(&c->full[tid], C::PAIR ? 2 : 1 + C::SF_UNITS);
            mbar_init(&c->sfull[tid], C::SF_UNITS > 0 ? C::SF_UNITS : 1);
            mbar_init(&c->empty[tid], 1);
        } else if (tid < C::STAGES + 2) {
            mbar_init(&c->dfull[tid - C::STAGES], 1);
            mbar_init(&c->dempty[tid - C::STAGES], (C::PAIR ? 2 : 1) * C::EPI);
        } else if (tid == 31) {
            mbar_init(&c->rfull, 1);
            mbar_init(&c->rempty, C::EPI * S);
            mbar_init(&c->fin, 1);
            c->abort = 0;
        }
        fence_mbar_init();
        __syncwarp();
    }
    if constexpr (C::PAIR) cluster_sync();   // both CTAs run and their barriers are ready
    if (warp == 1) tmem_alloc<C::PAIR>(&c->tmem, C::TMEM_COLS);
    if (!a.early) pdl_wait();
    pdl_launch_dependents();
    // tiles before each group: thread e (in rounds of the block) has group e, a scan within each
    // warp, then the warps' sums.  A group whose offsets do not lie in order within the rows is
    // recorded and left out.
    for (int e0 = 0, carry = 0; e0 < a.E; e0 += C::THREADS) {
        const int e = e0 + tid;
        int n = 0;
        if (e < a.E) {
            int rows = a.rows;
            if (a.offsets) {
                const int lo = a.offsets[e], hi = a.offsets[e + 1];
                rows = hi - lo;
                c->off[e] = lo;
                if (e == a.E - 1) c->off[a.E] = hi;
                if (lo < 0 || hi > a.rows || hi < lo) {
                    atomicOr(a.err, kErrBadOffsets);
                    rows = 0;
                }
            }
            n = mtiles * ((rows + a.width - 1) / a.width);
        }
        int sum = n;
#pragma unroll
        for (int d = 1; d < 32; d <<= 1) {
            const int o = __shfl_up_sync(0xffffffffu, sum, d);
            if (lane >= d) sum += o;
        }
        if (lane == 31) c->warp_tiles[warp] = sum;
        __syncthreads();
        int before = carry;
        for (int w = 0; w < C::THREADS / 32; ++w) {
            const int v = c->warp_tiles[w];
            if (w < warp) before += v;
            carry += v;
        }
        if (e < a.E) c->prefix[e] = before + sum - n;
        if (tid == 0) {
            c->prefix[a.E] = carry;   // the last round's stays
            c->tiles = carry;
        }
        __syncthreads();
    }
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    // Where ranks share a tile only the sums' exchange needs the others' barriers ready; the other
    // warps pass the cluster's barrier at the end.  (A pair's is behind it, and its stages are full only
    // with the peer's copies, which follow the peer's allocation.)
    if (!C::PAIR && S > 1) cluster_arrive();
    const uint32_t tmem = uniform(c->tmem);
    const int total = uniform(c->tiles);

    if (warp == 0 || warp == 3 || (C::NA == 2 && warp == 2)) {
        // ---------------- operands by TMA: one box of every stage ---------------------------
        const bool col = warp == 3;
        if (col && a.early) pdl_wait();
        const int o = warp >> 1;   // lanes operand
        const uint32_t to = smem_u32(ring) + (col ? C::NA : o) * C::A_BYTES;
        uint32_t it = 0;
        bool ok = true;
        for (int t = tile0; t < total && ok && !stopped(c); t += tstep) {
            const Tile q = get_tile<C>(a, c, t);
            const int cols = C::PAIR ? q.np >> 1 : q.np;   // this CTA's
            const uint32_t bytes = (C::PAIR ? 2u : 1u) * (C::NA * C::A_BYTES + (uint32_t)cols * 128u);
            const CUtensorMap *map = col ? &maps.b[(cols >> 4) - 1] : &maps.a[MODE == kMxMul2 ? 0 : o];
            const int y = col ? q.row0 + (C::PAIR ? rank * cols : 0) : q.e * a.M + q.m0 + lane0 + (MODE == kMxMul2 ? 2 * kM * o : 0);
            for (int ks = ks0; ks < ks1; ++ks, ++it) {
                const uint32_t s = it % C::STAGES;
                if (a.early && it == C::STAGES) pdl_wait();
                if (it >= C::STAGES && !(ok = wait_warp(&c->empty[s], ((it / C::STAGES) - 1) & 1, c, a.err))) break;
                const uint32_t bar = smem_u32(&c->full[s]), dst = to + s * (C::NA * C::A_BYTES + C::B_BYTES);
                if (warp == 0 && (!C::PAIR || rank == 0)) expect_tx(bar, bytes);
                if constexpr (C::PAIR) tma_2d_pair(dst, map, ks * (C::MX ? 128 : 64), y, map_rank(bar, 0));
                else tma_2d(dst, map, ks * (C::MX ? 128 : 64), y, bar);
            }
        }
        if (a.early) pdl_wait();
        // a pair: the leader's commits on the last stages' `empty`, which no load waits for, land before
        // this CTA ends and its shared memory is another kernel's
        if (C::PAIR && warp == 0)
            for (uint32_t j = it > (uint32_t)C::STAGES ? it - C::STAGES : 0; j < it && ok; ++j)
                ok = wait_warp(&c->empty[j % C::STAGES], (j / C::STAGES) & 1, c, a.err);
        __syncwarp();
    } else if (warp == 1 && !(C::PAIR && rank == 1)) {
        // ---------------- MMA issue ---------------------------------------------------------
        if (a.early) pdl_wait();
        const uint32_t r0 = smem_u32(ring), sf0 = smem_u32(sfring);
        uint32_t it = 0, h = 0;
        uint32_t gave = 0;   // bit i: the parity of half i's next wait; bit 2 + i: it has been used
        bool ok = true;
        for (int t = tile0; t < total && ok && !stopped(c); t += tstep) {
            const Tile q = get_tile<C>(a, c, t);
            const uint32_t idesc = a.idesc | (uint32_t)(q.np >> 3) << 17;
            const bool both = C::both_halves(q.np);
            if (both) h = 0;
            const uint32_t mine = both ? 3u : 1u << h;
            if ((mine & 1u) && (gave & 4u) && !(ok = wait_warp(&c->dempty[0], gave & 1u, c, a.err))) break;
            if ((mine & 2u) && (gave & 8u) && !(ok = wait_warp(&c->dempty[1], (gave >> 1) & 1u, c, a.err))) break;
            gave = (gave ^ (mine & (gave >> 2))) | mine << 2;   // the first use waits for nothing
            const uint32_t d0 = tmem + h * C::HALF, dstep = both ? BN : C::HALF / 2;
            for (int ks = ks0; ks < ks1; ++ks, ++it) {
                const uint32_t s = it % C::STAGES;
                if (!(ok = wait_warp(&c->full[s], (it / C::STAGES) & 1, c, a.err))) break;
                if (C::PAIR && !(ok = wait_warp(&c->sfull[s], (it / C::STAGES) & 1, c, a.err))) break;
                const uint32_t as = r0 + s * (C::NA * C::A_BYTES + C::B_BYTES), bs = as + C::NA * C::A_BYTES;
                uint32_t sfc = 0;
                if constexpr (C::MX) {
                    // the scales' TMEM buffer was last read by the MMAs of two stages ago
                    if (it >= 2 && !(ok = wait_warp(&c->empty[(it - 2) % C::STAGES], ((it - 2) / C::STAGES) & 1, c, a.err)))
                        break;
                    tc::fence_after_sync();
                    sfc = tmem + C::SF_COL + (it & 1) * C::SF_BUF;
                    const uint64_t sd = sdesc_scales(sf0 + s * C::SF_BYTES);
                    // columns: [block of 128 inputs][lanes operand 0, 1: 4 each, columns: 8]
#pragma unroll
                    for (int b = 0; b < 2; ++b) {
#pragma unroll
                        for (int u = 0; u < C::SF_UNITS; ++u) {
                            const uint32_t to = sfc + b * 16 + (u < C::NA ? u * 4 : 8 + (u - C::NA) * 4);
                            const uint64_t from = sd + (uint64_t)((u * 1024 + b * 512) >> 4);
                            if constexpr (C::PAIR) cp_scales_pair(to, from);
                            else cp_scales(to, from);
                        }
                    }
                } else {
                    tc::fence_after_sync();
                }
                const uint64_t bd = tc::sdesc_kmajor_sw128(bs);
#pragma unroll
                for (int k = 0; k < 4; ++k) {
#pragma unroll
                    for (int o = 0; o < C::NA; ++o) {
                        const uint64_t ka = tc::sdesc_kmajor_sw128(as + o * C::A_BYTES) + k * 2, kb = bd + k * 2;
                        if constexpr (C::MX) {
                            const uint32_t id = idesc | (uint32_t)((k & 1) * 2) << 29 | (uint32_t)((k & 1) * 2) << 4;
                            const uint32_t sa = sfc + (k >> 1) * 16 + o * 4, sb = sfc + (k >> 1) * 16 + 8;
                            if constexpr (C::PAIR) mma_mx4_pair(d0 + o * dstep, ka, kb, id, sa, sb, ks > ks0 || k > 0);
                            else mma_mx4(d0 + o * dstep, ka, kb, id, sa, sb, ks > ks0 || k > 0);
                        } else {
                            mma_f16(d0 + o * dstep, ka, kb, idesc, ks > ks0 || k > 0);
                        }
                    }
                }
                commit<C::PAIR>(&c->empty[s]);
            }
            commit<C::PAIR>(&c->dfull[h]);
            if (both) commit<C::PAIR>(&c->dfull[1]);
            else h ^= 1;
        }
        commit<C::PAIR>(&c->fin);   // every MMA issued here is done before TMEM is freed
    } else if (C::PAIR && warp == 1) {
        // ---------------- the peer's scales: one word a stage to the leader ------------------
        // The warps that wrote the scales have made them visible to the tensor unit (the async proxy)
        // before they arrived here; the word goes out as a commit of no operations, which costs
        // the warp little.  (An ordinary arrival with release at cluster scope took about 1500
        // cycles a stage from here, 2000 from the warps that load the scales.)
        if (a.early) pdl_wait();
        uint32_t it = 0;
        bool ok = true;
        for (int t = tile0; t < total && ok && !stopped(c); t += tstep)
            for (int ks = ks0; ks < ks1; ++ks, ++it) {
                const uint32_t s = it % C::STAGES;
                if (!(ok = wait_warp(&c->sfull[s], (it / C::STAGES) & 1, c, a.err))) break;
                commit_leader(&c->full[s]);
            }
    } else if (warp >= 4 && warp < 4 + C::EPI) {
        // ---------------- epilogue: 32 lanes, 16 columns at a time; two warps take turns ----
        if (!C::PAIR && S > 1) cluster_wait();
        if (a.early) pdl_wait();
        const int qd = warp & 3, part = (warp - 4) >> 2;
        const uint32_t tl = tmem + ((uint32_t)(qd * 32) << 16);
        uint32_t nt = 0, h = 0, red_parity = 0, parity = 0;   // parity: bit i of half i's next wait
        bool ok = true;
        for (int t = tile0; t < total && ok && !stopped(c); t += tstep, ++nt) {
            const Tile q = get_tile<C>(a, c, t);
            const int m = q.m0 + lane0 + qd * 32 + lane;
            const bool both = C::both_halves(q.np);
            if (both) h = 0;
            const uint32_t mine = both ? 3u : 1u << h;   // the tile's halves
            if ((mine & 1u) && !(ok = wait_warp(&c->dfull[0], parity & 1u, c, a.err))) break;
            if ((mine & 2u) && !(ok = wait_warp(&c->dfull[1], (parity >> 1) & 1u, c, a.err))) break;
            parity ^= mine;
            tc::fence_after_sync();
            const uint32_t d0 = tl + h * C::HALF, dstep = both ? BN : C::HALF / 2;
            if (!both) h ^= 1;
            if (C::FEW && S > 1) {
                // send the partial sums to their columns' owners (column k to rank k % S), then
                // add up the own columns in rank order
                // the buffers are used again: the host gives every tile a cluster of its own, but lists
                // out of order can name rows more than once and hold more tiles than it counts
                const bool more = t + tstep < total;
                const int per = (kSplitCols + S - 1) / S, own = q.n > rank ? (q.n - rank + S - 1) / S : 0;
                if (warp == 4 && lane == 0 && own > 0)
                    mbar_arrive_expect_tx(&c->rfull, (uint32_t)(S * own * C::NA * kM * 4));
                if (nt >= 1 && !(ok = wait_warp_cluster(&c->rempty, (nt - 1) & 1, c, a.err))) break;
                const uint32_t mine0 = smem_u32(red) + (uint32_t)((rank * per * kM + qd * 32 + lane) * 4);
                const uint32_t rbar = smem_u32(&c->rfull);
                for (int k = 0, owner = 0, slot = 0; k < q.n; ++k) {
                    uint32_t v[2];
                    ld1<C::NA>(d0 + k, dstep, v);
                    const uint32_t bar = map_rank(rbar, owner);
#pragma unroll
                    for (int o = 0; o < C::NA; ++o)
                        st_async(map_rank(mine0 + (uint32_t)((o * C::RED_COLS + slot) * kM * 4), owner), v[o], bar);
                    if (++owner == S) {
                        owner = 0;
                        ++slot;
                    }
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->dempty[mine >> 1]);   // tiles of this form take one half
                if (own > 0) {
                    if (!(ok = wait_warp_cluster(&c->rfull, red_parity, c, a.err))) break;
                    red_parity ^= 1;
                    for (int i = 0; i < own; ++i) {
                        float x[2] = {0.0f, 0.0f};
                        for (int r = 0; r < S; ++r)
#pragma unroll
                            for (int o = 0; o < C::NA; ++o) x[o] += red[(o * C::RED_COLS + r * per + i) * kM + qd * 32 + lane];
                        emit1<MODE>(a, x[0], x[1], m, lane, q.row0 + i * S + rank);
                    }
                }
                __syncwarp();
                if (more && lane < S) arrive_cluster(map_rank(smem_u32(&c->rempty), lane));
            } else if (C::FEW) {
                for (int k = 0; k < q.n; ++k) {
                    __syncwarp();   // lanes past M come from another branch, the load wants the whole warp
                    uint32_t v[2];
                    ld1<C::NA>(d0 + k, dstep, v);
                    emit1<MODE>(a, __uint_as_float(v[0]), __uint_as_float(v[1]), m, lane, q.row0 + k);
                }
                tc::fence_before_sync();
                __syncwarp();
                if (lane == 0) mbar_arrive(&c->dempty[mine >> 1]);
            } else {
                // the accumulators go back to the pair's leader once this warp has read its part
                const auto give_back = [&] {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0 && (mine & 1u)) arrive_cluster_relaxed(map_rank(smem_u32(&c->dempty[0]), 0));
                    if (lane == 0 && (mine & 2u)) arrive_cluster_relaxed(map_rank(smem_u32(&c->dempty[1]), 0));
                };
                if (part * 16 >= q.np) give_back();
                for (int c0 = part * 16; c0 < q.np; c0 += 4 * C::EPI) {
                    __syncwarp();   // as above
                    uint32_t v[2][16];
#pragma unroll
                    for (int o = 0; o < C::NA; ++o) tc::ld16(d0 + o * dstep + c0, v[o]);
                    tc::wait_ld();
                    float f[2][16];
#pragma unroll
                    for (int o = 0; o < C::NA; ++o)
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            asm volatile("" : "+r"(v[o][j]));   // read after the wait
                            f[o][j] = __uint_as_float(v[o][j]);
                        }
                    if (c0 + 4 * C::EPI >= q.np) give_back();
                    emit16<MODE>(a, f[0], f[C::NA - 1], m, lane,
                                 [&](int j) { return c0 + j < q.n ? q.row0 + c0 + j : -1; });
                }
            }
        }
    } else if (C::MX && warp >= C::SF_WARP) {
        // ---------------- scales: this warp's operand, 128 rows -----------------------------
        // Chunks of 512 inputs (16 scale bytes of a row, two stages), one ahead in registers, over
        // the tiles' ends too.  The next chunk is loaded before this one is stored where the MMAs
        // set the pace (prompt 1255 us, after: 1276), after it where the weights' stream does (decode
        // batch 486 us, before: 502), but for rows off the 16-byte grid, which have more to load
        // (decode batch of 4160 x 1088 75 us, after: 80).  Further ahead is slower (prompt block 969 us,
        // two chunks 980, four 1133): the fence before the arrival waits for a warp's loads in flight.
        const int u = warp - C::SF_WARP;
        if (u >= C::NA && a.early) pdl_wait();
        const uint8_t *base = u < C::NA ? a.sfa[MODE == kMxMul2 ? 0 : u] : a.sfb;
        const long long rows = u < C::NA ? a.sfa_rows : a.rows;
        const int kc0 = ks0 >> 1, kc1 = (ks1 + 1) >> 1;
        const int chunks = tile0 < total ? (total - tile0 + tstep - 1) / tstep * (kc1 - kc0) : 0;
        int lt = tile0 - tstep, lk = kc1;   // the next load: tile, chunk
        long long lrow = 0;
        Scales<WHOLE> v[4];
        auto load = [&] {
            if (lk == kc1) {
                lt += tstep;
                lk = kc0;
                if (lt < total) {
                    const Tile q = get_tile<C>(a, c, lt);
                    lrow = u < C::NA ? (long long)q.e * a.M + q.m0 + lane0 + (MODE == kMxMul2 ? 2 * kM * u : 0) : (long long)q.row0 + (u - C::NA) * 128;
                }
            }
            if (lt < total) {
#pragma unroll
                for (int i = 0; i < 4; ++i) v[i].load(base, lrow + lane + 32 * i, rows, a.sf_ld, lk);
                ++lk;
            }
        };
        load();
        uint32_t it = 0;
        int kc = kc0;
        bool ok = true;
        for (int i = 0; i < chunks && ok; ++i) {
            uint4 now[4];
#pragma unroll
            for (int j = 0; j < 4; ++j) now[j] = v[j].get();
            if (!C::FEW || !WHOLE || i == 0) load();
            for (int ks = max(ks0, 2 * kc); ks < min(ks1, 2 * kc + 2); ++ks, ++it) {
                const uint32_t s = it % C::STAGES;
                if (a.early && it == C::STAGES) pdl_wait();
                if (it >= C::STAGES && !(ok = wait_warp(&c->empty[s], ((it / C::STAGES) - 1) & 1, c, a.err))) break;
                uint4 *dst = reinterpret_cast<uint4 *>(sfring + s * C::SF_BYTES + u * 1024) + lane;
                const bool odd = ks & 1;
                dst[0] = make_uint4(odd ? now[0].z : now[0].x, odd ? now[1].z : now[1].x, odd ? now[2].z : now[2].x, odd ? now[3].z : now[3].x);
                dst[32] = make_uint4(odd ? now[0].w : now[0].y, odd ? now[1].w : now[1].y, odd ? now[2].w : now[2].y, odd ? now[3].w : now[3].y);
                tc::fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) mbar_arrive(C::PAIR ? &c->sfull[s] : &c->full[s]);
            }
            if (C::FEW && WHOLE && i > 0) load();
            if (++kc == kc1) kc = kc0;
        }
    }

    if (!C::PAIR && S > 1 && !(warp >= 4 && warp < 4 + C::EPI)) cluster_wait();
    if (a.early) pdl_wait();   // a CTA without tiles too: this grid ends after the one before it
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 1) settle(&c->fin, &c->abort);   // (a pair: the leader's last commit, in both CTAs)
    // no CTA of a cluster frees its TMEM or leaves while another may still use its memory
    if (CS > 1) cluster_sync();
    if (warp == 1) {
        tc::fence_after_sync();
        tmem_dealloc<C::PAIR>(tmem, C::TMEM_COLS);
        __syncwarp();
    }
    if (C::PAIR) cluster_sync();
}

// Clusters of `size` CTAs of this kernel that the current device holds at once (0 if unknown); a
// cluster lies within one of the device's processor groups, so this is less than SMs / size
// (measured on GB300 with one CTA an SM: 76, 46, 36, 28, 23, 15, 15 for 2 to 8).
template <Mode MODE, int BN, bool WHOLE>
int max_clusters(int size)
{
    static std::atomic<int> known[64][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][size].load();
    if (n == 0) {
        cudaLaunchConfig_t cfg = {};
        cfg.gridDim = dim3(size * num_sms());
        cfg.blockDim = dim3(Cfg<MODE, BN>::THREADS);
        cfg.dynamicSmemBytes = Cfg<MODE, BN>::SMEM;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = (unsigned)size;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        const void *k = reinterpret_cast<const void *>(gemm_kernel<MODE, BN, WHOLE>);
        if (ensure_dynamic_smem(k, Cfg<MODE, BN>::SMEM) != cudaSuccess ||
            cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
            cudaGetLastError();
            return 0;
        }
        known[dev][size].store(n);
    }
    return n;
}

// CTAs that share a tile when `tiles` of them would leave SMs idle: each with two stages of the
// reduction at least, with eight where a quarter of the SMs has a tile anyway (48 tiles of 8 stages
// 5.4 us alone, 5.9 by threes; one token, microseconds with at least 8, 4, 2 stages a CTA: 16-bit block of
// 1000 x 520 6.6, 5.1, 4.5, of 2048 x 512 5.4, 4.6, 4.6; MXFP4 product of 16 rows, 1000 x 4096 7.8,
// 5.8, 5.1).  All clusters run at once: the query counts one CTA an SM, PER_SM fit.
template <Mode MODE, int BN, bool WHOLE>
int choose_split(long long tiles, int ksteps)
{
    int best = 1;
    if (Cfg<MODE, BN>::FEW)
        for (int s = 2; s <= 8 && (4 * tiles > num_sms() ? 8 : 2) * s <= ksteps && s * tiles <= num_sms(); ++s)
            if (Cfg<MODE, BN>::PER_SM * max_clusters<MODE, BN, WHOLE>(s) >= tiles) best = s;
    return best;
}

template <Mode MODE, int BN, bool WHOLE>
cudaError_t launch(const Args &a, const Maps &m, int grid, cudaStream_t st)
{
    using C = Cfg<MODE, BN>;
    return launch_kernel(gemm_kernel<MODE, BN, WHOLE>, dim3(grid), dim3(C::THREADS), C::SMEM, st, C::PAIR ? 2 : a.split, a, m);
}

}  // namespace gemm
}  // namespace moe
