// adapter_tiles.cuh -- adapters on tiles of 128 rows of one segment, both products on tcgen05, in two kernels:
//
//   u = x down^T.  A cluster of up to 8 CTAs takes a tile (128 rows on the accumulator's lanes, the rank in its
//   columns), each CTA a share of the inputs; the shares are added in rank order through distributed shared
//   memory.  u goes to the workspace in 16-bit parts, each what the ones before it leave: three of bf16 where y is
//   fp32, 2^-24 of the number at most, and otherwise two, 2^-17 in bf16 (for a y of 16 bits, whose own rounding
//   takes 2^-9 or 2^-12) and 2^-22 of the row's largest in fp16, which has it brought to 2^13 (so as neither to
//   overflow nor to lose the last part to the smallest numbers) and its sums brought back before the adapter's factor.
//   y = base + scale u up^T.  A CTA takes a tile and a run of output columns, 128 bytes of a row at a time: u
//   stays in its shared memory, up and base come by TMA, and a thread of the epilogue adds 64 consecutive bytes
//   of a row and stores them.  Two parts' products cost nothing beside the memory; a third takes 0 to 5 % at ranks up
//   to 64 (8192 rows, 6144 x 6144, rank 64, fp32 y: 98 to 101 us; one row 10.2 to 11.2) and up to 15 % at 128, where
//   it leaves the ring 5 stages for 6 (3000 rows 57 to 65).
//
// What they move is x once and base and y once: bound by memory.  Two CTAs stand on an SM (half of its shared
// memory each) with a ring of copies in flight.  One kernel for both products, the clusters handing u on
// through distributed shared memory, was slower: 105 us where these take 67 (8192 rows, 6144 x 6144, rank 64):
// every tile's exchange, 15,000 cycles, stood between its two streams.
//
// Warps: 0 and 1 load (x and down; base and up), 2 issues the MMAs, those from 4 on are the epilogue.  Every wait
// is bounded (cluster_wait.cuh); every thread goes to every cluster barrier.
#pragma once

#include <algorithm>
#include <atomic>
#include <type_traits>

#include "adapter.cuh"
#include "gemm_tc.cuh"
#include "tensor_map.cuh"

namespace moe {
namespace adapter {

using gemm::expect_tx;
using gemm::tma_2d;
using gemm::uniform;

constexpr int kTileRows = 128;
constexpr int kFirstEpi = 4;
constexpr int kDownThreads = 32 * (kFirstEpi + 4), kUpThreads = 32 * (kFirstEpi + 8);
constexpr int kMaxTileStages = 8;
constexpr int kXBytes = kTileRows * 128;
constexpr int kTmemCols = 128, kUpStep = 64;
constexpr int kHalfSm = 112 * 1024;   // shared memory of a CTA where two stand on an SM
constexpr int kMaxParts = 3;
// fp32's range is bf16's, but not fp16's
template <typename T>
constexpr bool kBroughtUp = std::is_same<T, __half>::value;

struct TileArgs {
    AdapterArgs p;
    int row0, cell0, cell1;   // rows and grid cells of this pass
    int r16;             // rank in steps of 16
    int blocks;          // of 64 ranks
    int ksteps, splits;  // down: stages of 64 inputs in all, CTAs that share them
    int chunks, slices;  // up: of the outputs' columns, CTAs of a tile
    int stages, stage_bytes;
    uint32_t idesc;      // without N
    int parts;           // of a value of u
    void *u[kMaxParts];  // [rows of the pass][r16]
    float *back;         // fp16: what undoes a row's scaling
    int wide;            // y's rows lie on 32-byte boundaries
};

// operands with a row a tile's row: boxes of all 128, and of 32 for a tile that has no more (its other lanes
// hold whatever was there; none of them is stored)
constexpr int kShortRows = 32;
struct TileMaps {
    CUtensorMap a[2], b, u[kMaxParts][2];   // x, down | base, up, u's parts
};

struct TileCtrl {
    uint64_t full[kMaxTileStages], empty[kMaxTileStages], ufull, dfull[2], dempty[2], fin;
    uint32_t tmem;
    int abort;
    Tile tile;
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void store64(char *p, const uint32_t (&w)[16], int n, bool wide)
{
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        if (wide && i + 1 < n) {
            asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p + 16 * i), "r"(w[4 * i]), "r"(w[4 * i + 1]),
                         "r"(w[4 * i + 2]), "r"(w[4 * i + 3]), "r"(w[4 * i + 4]), "r"(w[4 * i + 5]), "r"(w[4 * i + 6]), "r"(w[4 * i + 7])
                         : "memory");
        } else {
#pragma unroll
            for (int j = i; j < i + 2; ++j)
                if (j < n) *reinterpret_cast<uint4 *>(p + 16 * j) = make_uint4(w[4 * j], w[4 * j + 1], w[4 * j + 2], w[4 * j + 3]);
        }
    }
}

// had + scale * (back * v) of consecutive columns, in place
template <typename Y, bool BACK>
__device__ __forceinline__ void add_columns(uint32_t (&w)[sizeof(Y) * 4], const uint32_t (&v)[16], float scale, float back)
{
    union {
        uint32_t w;
        Y y[4 / sizeof(Y)];
    } u;
    constexpr int N = 4 / sizeof(Y);
#pragma unroll
    for (int i = 0; i < 16 / N; ++i) {
        u.w = w[i];
#pragma unroll
        for (int j = 0; j < N; ++j) {
            const float sum = __uint_as_float(v[i * N + j]);
            from_f32(u.y[j], fmaf(scale, BACK ? back * sum : sum, to_f32(u.y[j])));
        }
        w[i] = u.w;
    }
}

// the ring of copies, as one warp goes through it
struct Turn {
    uint32_t it = 0, s = 0, phase = 0;
    __device__ __forceinline__ void next(int stages)
    {
        ++it;
        if (++s == (uint32_t)stages) {
            s = 0;
            phase ^= 1;
        }
    }
};

// barriers, tensor memory and this CTA's tile; the caller's kernel may read what the kernel before it wrote
// where `after` is set
__device__ __forceinline__ void set_up(const TileArgs &a, TileCtrl *c, int number, uint32_t empties, uint32_t epilogue, bool after)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (warp == 0) {
        if (tid < kMaxTileStages) {
            mbar_init(&c->full[tid], 1);
            mbar_init(&c->empty[tid], empties);
        } else if (tid < kMaxTileStages + 2) {
            mbar_init(&c->dfull[tid - kMaxTileStages], 1);
            mbar_init(&c->dempty[tid - kMaxTileStages], epilogue);
        } else if (tid == 31) {
            mbar_init(&c->ufull, 1);
            mbar_init(&c->fin, 1);
            c->abort = 0;
        }
        fence_mbar_init();
        __syncwarp();
        if (after) pdl_wait();
        const Tile t = find_tile(a.p, number, kTileRows, lane);
        if (lane == 0) {
            c->tile = t;
            if (t.lo < t.hi && (t.lo / kTileRows < a.cell0 || t.lo / kTileRows >= a.cell1)) c->tile.hi = c->tile.lo;   // another pass's
        }
    }
    if (warp == 2) gemm::tmem_alloc<false>(&c->tmem, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    if (after) {
        pdl_wait();
        pdl_launch_dependents();
    }
}

template <typename T>
__global__ void __launch_bounds__(kDownThreads, 2) adapter_down_kernel(const __grid_constant__ TileArgs a, const __grid_constant__ TileMaps maps)
{
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    TileCtrl *c = reinterpret_cast<TileCtrl *>(ring + a.stages * a.stage_bytes);
    const AdapterArgs &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const int rank = blockIdx.x % a.splits, index = blockIdx.x / a.splits;
    set_up(a, c, a.cell0 + index, 1, 1, true);
    if (rank == 0 && tid == 0 && a.cell0 == 0 && index < p.S) check_segment(p, index);
    const uint32_t tmem = uniform(c->tmem);
    const Tile t = c->tile;
    if (t.lo >= t.hi || t.adapter < 0 || t.bad) {   // (the same for the whole cluster)
        if (warp == 2) gemm::tmem_dealloc<false>(tmem, kTmemCols);
        return;
    }
    const int kper = (a.ksteps + a.splits - 1) / a.splits;
    const int k0 = min(a.ksteps, rank * kper), ksteps = min(a.ksteps, k0 + kper) - k0;
    const uint32_t r0 = smem_u32(ring);
    const bool few = t.hi - t.lo <= kShortRows;
    const auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, &c->abort, p.err); };
    const int pitch = p.R + 4;   // of the rows' sums, which take the ring's place
    Turn at;
    bool ok = true;
    if (warp <= 1) {
        const int y = warp == 0 ? uniform(t.lo) : uniform(t.adapter) * p.R;
        const CUtensorMap *map = warp == 0 ? &maps.a[few] : &maps.b;
        const uint32_t bytes = (few ? kShortRows : kTileRows) * 128 + a.r16 * 128;
        for (int k = 0; k < ksteps; ++k, at.next(a.stages)) {
            if (at.it >= (uint32_t)a.stages && !(ok = wait(&c->empty[at.s], at.phase ^ 1))) break;
            const uint32_t bar = smem_u32(&c->full[at.s]);
            if (warp == 0) expect_tx(bar, bytes);
            tma_2d(r0 + at.s * a.stage_bytes + (warp == 0 ? 0 : kXBytes), map, 64 * (k0 + k), y, bar);
        }
        if (warp == 0)   // the last commits land before this shared memory is another kernel's
            for (uint32_t j = at.it > (uint32_t)a.stages ? at.it - a.stages : 0; j < at.it && ok; ++j)
                ok = wait(&c->empty[j % a.stages], (j / a.stages) & 1);
    } else if (warp == 2) {
        const uint32_t idesc = a.idesc | (uint32_t)(a.r16 >> 3) << 17;
        for (int k = 0; k < ksteps; ++k, at.next(a.stages)) {
            if (!(ok = wait(&c->full[at.s], at.phase))) break;
            tc::fence_after_sync();
            const uint32_t from = r0 + at.s * a.stage_bytes;
            const uint64_t xd = tc::sdesc_kmajor_sw128(from), dd = tc::sdesc_kmajor_sw128(from + kXBytes);
#pragma unroll
            for (int j = 0; j < 4; ++j) gemm::mma_f16(tmem, xd + 2 * j, dd + 2 * j, idesc, k > 0 || j > 0);
            tc::commit_elect(&c->empty[at.s]);
        }
        tc::commit_elect(&c->ufull);
    } else if (warp >= kFirstEpi) {
        ok = wait(&c->ufull, 0);   // (every product has read the ring)
        tc::fence_after_sync();
        float *to = reinterpret_cast<float *>(ring) + ((warp & 3) * 32 + lane) * pitch;
        for (int r = 0; r < a.r16; r += 16) {
            uint32_t v[16];
            tc::ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + r, v);
            tc::wait_ld();
#pragma unroll
            for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));   // read after the wait
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (r + i < p.R)
                    *reinterpret_cast<uint4 *>(to + r + i) = ksteps > 0 ? make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]) : make_uint4(0, 0, 0, 0);
        }
        tc::fence_before_sync();
    }
    __syncwarp();
    cluster_sync();   // every CTA's sums are there
    // this CTA's share of the rows: added over the cluster, two rows of a warp at a time, and cut into 16-bit parts
    constexpr int kWarps = kDownThreads / 32, kAtOnce = 2;
    const int rows = min(kTileRows / a.splits, t.hi - t.lo - rank * (kTileRows / a.splits));
    for (int i0 = warp; i0 < rows; i0 += kWarps * kAtOnce) {
        float4 w[kAtOnce][8];
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            if (i0 + n * kWarps >= rows) continue;   // nothing is read that is not used: the barrier at the end waits for no read
            const int row = rank * (kTileRows / a.splits) + i0 + n * kWarps;
            const uint32_t from = r0 + (uint32_t)(row * pitch + 4 * lane) * 4;
            if (4 * lane < p.R)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < a.splits) w[n][q] = ld_cluster_v4(map_rank(from, q));
        }
#pragma unroll
        for (int n = 0; n < kAtOnce; ++n) {
            if (i0 + n * kWarps >= rows) continue;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (4 * lane < p.R)
#pragma unroll
                for (int q = 0; q < 8; ++q)
                    if (q < a.splits) {
                        v[0] += w[n][q].x;
                        v[1] += w[n][q].y;
                        v[2] += w[n][q].z;
                        v[3] += w[n][q].w;
                    }
            const size_t line = (size_t)(t.lo + rank * (kTileRows / a.splits) + i0 + n * kWarps - a.row0);
            if constexpr (kBroughtUp<T>) {
                float top = 0.0f;
                bool odd = false;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    top = fmaxf(top, fabsf(v[j]));
                    odd |= !(fabsf(v[j]) <= 3.4e38f);
                }
                const uint32_t bits = __reduce_max_sync(0xffffffffu, __float_as_uint(top));
                int shift = bits == 0 ? 0 : 13 - ((int)(bits >> 23) - 127);
                if (__any_sync(0xffffffffu, odd)) shift = 0;   // infinities and NaN stay what they are
                shift = max(-126, min(126, shift));
                const float by = __uint_as_float((uint32_t)(shift + 127) << 23);
#pragma unroll
                for (int j = 0; j < 4; ++j) v[j] *= by;
                if (lane == 0) a.back[line] = __uint_as_float((uint32_t)(127 - shift) << 23);
            }
#pragma unroll
            for (int i = 0; i < kMaxParts; ++i) {
                if (i == a.parts) break;
                union {
                    uint2 w;
                    T t[4];
                } part;
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    from_f32(part.t[j], v[j]);
                    const float had = to_f32(part.t[j]);
                    v[j] = fabsf(had) <= 3.4e38f ? v[j] - had : 0.0f;
                }
                if (4 * lane < a.r16) *reinterpret_cast<uint2 *>(static_cast<T *>(a.u[i]) + line * a.r16 + 4 * lane) = part.w;
            }
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        settle(&c->ufull, &c->abort);
        tc::fence_after_sync();
        gemm::tmem_dealloc<false>(tmem, kTmemCols);
        __syncwarp();
    }
    // no CTA leaves while another reads its sums (or, once it has given up, writes to its memory)
    if (aborted(&c->abort)) cluster_sync();
    else cluster_sync_relaxed();
}

template <typename T, typename Y>
__global__ void __launch_bounds__(kUpThreads, 2) adapter_up_kernel(const __grid_constant__ TileArgs a, const __grid_constant__ TileMaps maps)
{
    constexpr int CW = 64 / sizeof(Y);   // columns of a thread
    constexpr int NC = 2 * CW;           // of a chunk
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *ubuf = ring + a.stages * a.stage_bytes;   // part by part
    TileCtrl *c = reinterpret_cast<TileCtrl *>(ubuf + a.parts * a.blocks * kXBytes);
    const AdapterArgs &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const int slice = blockIdx.x % a.slices, index = blockIdx.x / a.slices;
    // lists, base and up are older than the kernel before this one, which waited for them
    set_up(a, c, a.cell0 + index, 9, 8, false);
    const uint32_t tmem = uniform(c->tmem);
    const Tile t = c->tile;
    const int per = (a.chunks + a.slices - 1) / a.slices;
    const int chunk0 = min(a.chunks, slice * per), nchunks = min(a.chunks, chunk0 + per) - chunk0;
    if (t.lo >= t.hi || t.adapter < 0 || t.bad || nchunks == 0) {
        pdl_wait();
        pdl_launch_dependents();
        if (t.lo < t.hi && (t.adapter < 0 || t.bad) && nchunks > 0)
            pass_through<Y>(p, t, chunk0 * NC, min(p.N, (chunk0 + nchunks) * NC), tid, kUpThreads);
        if (warp == 2) gemm::tmem_dealloc<false>(tmem, kTmemCols);
        return;
    }
    const uint32_t r0 = smem_u32(ring), u0 = smem_u32(ubuf);
    const int adapter = uniform(t.adapter), row0 = uniform(t.lo);
    const bool few = t.hi - t.lo <= kShortRows;
    const int row_bytes = (few ? kShortRows : kTileRows) * 128;   // of a box
    const auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, &c->abort, p.err); };
    Turn at;
    bool ok = true;
    if (warp == 0) {
        const uint32_t bytes = (p.base ? row_bytes : 0) + a.blocks * NC * 128;
        for (int j = 0; j < nchunks; ++j, at.next(a.stages)) {
            if (j == a.stages) pdl_wait();   // (no bounded wait begins before the kernel ahead ends)
            if (j >= a.stages && !(ok = wait(&c->empty[at.s], at.phase ^ 1))) break;
            const uint32_t bar = smem_u32(&c->full[at.s]);
            expect_tx(bar, bytes);
            if (p.base) tma_2d(r0 + at.s * a.stage_bytes, &maps.a[few], 64 * (chunk0 + j), row0, bar);   // 128 bytes, of whatever type
        }
        pdl_wait();
        for (uint32_t j = at.it > (uint32_t)a.stages ? at.it - a.stages : 0; j < at.it && ok; ++j)
            ok = wait(&c->empty[j % a.stages], (j / a.stages) & 1);
    } else if (warp == 1) {
        for (int j = 0; j < nchunks; ++j, at.next(a.stages)) {
            if (j == a.stages) pdl_wait();
            if (j >= a.stages && !(ok = wait(&c->empty[at.s], at.phase ^ 1))) break;
            for (int b = 0; b < a.blocks; ++b)
                tma_2d(r0 + at.s * a.stage_bytes + kXBytes + b * NC * 128, &maps.b, 64 * b, adapter * p.N + (chunk0 + j) * NC, smem_u32(&c->full[at.s]));
        }
        pdl_wait();
    } else if (warp == 3) {
        pdl_wait();
        pdl_launch_dependents();
        const uint32_t bar = smem_u32(&c->ufull);
        expect_tx(bar, a.parts * a.blocks * row_bytes);
        for (int i = 0; i < a.parts; ++i)
            for (int b = 0; b < a.blocks; ++b) tma_2d(u0 + (i * a.blocks + b) * kXBytes, &maps.u[i][few], 64 * b, row0 - a.row0, bar);
    } else if (warp == 2) {
        const uint32_t idesc = a.idesc | (uint32_t)(NC >> 3) << 17;
        pdl_wait();
        ok = wait(&c->ufull, 0);
        for (int j = 0; j < nchunks && ok; ++j, at.next(a.stages)) {
            const uint32_t buf = j & 1, use = j >> 1, d = tmem + buf * kUpStep;
            if (use >= 1 && !(ok = wait(&c->dempty[buf], (use - 1) & 1))) break;
            if (!(ok = wait(&c->full[at.s], at.phase))) break;
            tc::fence_after_sync();
            uint32_t first = 0;
            for (int part = 0; part < a.parts; ++part)
                for (int k = 0; k < a.r16; k += 16) {
                    const uint64_t ud = tc::sdesc_kmajor_sw128(u0 + (part * a.blocks + (k >> 6)) * kXBytes) + ((k & 63) >> 3);
                    const uint64_t wd = tc::sdesc_kmajor_sw128(r0 + at.s * a.stage_bytes + kXBytes + (k >> 6) * NC * 128) + ((k & 63) >> 3);
                    gemm::mma_f16(d, ud, wd, idesc, first);
                    first = 1;
                }
            tc::commit_elect(&c->empty[at.s]);
            tc::commit_elect(&c->dfull[buf]);
        }
        tc::commit_elect(&c->fin);
    } else {
        pdl_wait();
        const int part = (warp - kFirstEpi) >> 2, local = (warp & 3) * 32 + lane, row = t.lo + local;
        const bool on = row < t.hi;
        const float scale = p.scale ? p.scale[adapter] : 1.0f, back = kBroughtUp<T> && on ? a.back[row - a.row0] : 1.0f;
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + part * CW;
        char *line = static_cast<char *>(p.y) + ((size_t)row * p.N + part * CW) * sizeof(Y);
        for (int j = 0; j < nchunks; ++j, at.next(a.stages)) {
            const uint32_t buf = j & 1, use = j >> 1;
            uint32_t w[16];
            if (!(ok = wait(&c->full[at.s], at.phase))) break;
            if (p.base) {
                const uint8_t *from = ring + at.s * a.stage_bytes + local * 128;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(from + (((part * 4 + i) ^ (local & 7)) << 4));
                    w[4 * i] = v.x;
                    w[4 * i + 1] = v.y;
                    w[4 * i + 2] = v.z;
                    w[4 * i + 3] = v.w;
                }
                tc::fence_proxy_async_smem();   // these reads come before the next copy into the stage
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) w[i] = 0;
            }
            __syncwarp();
            if (lane == 0) mbar_arrive(&c->empty[at.s]);
            if (!(ok = wait(&c->dfull[buf], use & 1))) break;
            tc::fence_after_sync();
#pragma unroll
            for (int h = 0; h < CW; h += 16) {
                uint32_t v[16];
                tc::ld16(tl + buf * kUpStep + h, v);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));
                if (h + 16 == CW) {
                    tc::fence_before_sync();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&c->dempty[buf]);
                }
                constexpr int W = sizeof(Y) * 4;   // words of 16 columns
                add_columns<Y, kBroughtUp<T>>(*reinterpret_cast<uint32_t(*)[W]>(&w[h / 16 * W]), v, scale, back);
            }
            const int n = (chunk0 + j) * NC;
            if (on) store64(line + (size_t)n * sizeof(Y), w, (p.N - n - part * CW) / (CW / 4), a.wide);
            __syncwarp();
        }
    }
    __syncwarp();
    tc::fence_before_sync();
    __syncthreads();
    if (warp == 2) {
        settle(&c->fin, &c->abort);
        tc::fence_after_sync();
        gemm::tmem_dealloc<false>(tmem, kTmemCols);
        __syncwarp();
    }
}

// bytes of the workspace for a row of a pass
inline size_t row_bytes(int R) { return (size_t)(R + 15) / 16 * 16 * 2 * kMaxParts + 4; }

// clusters of `size` CTAs of the first kernel that the current device runs at once, two CTAs an SM (the query counts one)
template <typename T>
int down_clusters(int size)
{
    static std::atomic<int> known[64][9];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return 0;
    int n = known[dev][size].load();
    if (n) return n;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(size * num_sms());
    cfg.blockDim = dim3(kDownThreads);
    cfg.dynamicSmemBytes = kHalfSm;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)size;
    at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    const void *k = reinterpret_cast<const void *>(adapter_down_kernel<T>);
    if (ensure_dynamic_smem(k, kHalfSm) != cudaSuccess || cudaOccupancyMaxActiveClusters(&n, k, &cfg) != cudaSuccess) {
        cudaGetLastError();
        return 0;
    }
    known[dev][size].store(2 * n);
    return 2 * n;
}

template <typename T, typename Y>
cudaError_t launch_pass(TileArgs a, int dtype, cudaStream_t st)
{
    constexpr int NC = 128 / sizeof(Y);
    const AdapterArgs &p = a.p;
    const int tiles = a.cell1 - a.cell0 + p.S, slots = 2 * num_sms();
    const uint32_t f = dtype == MOE_DTYPE_BF16 ? 1u : 0u;
    a.idesc = (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)(kTileRows >> 4) << 24);
    a.r16 = (p.R + 15) / 16 * 16;
    a.blocks = (p.R + 63) / 64;
    const int rows = std::min(p.T - a.row0, (a.cell1 - a.cell0) * kTileRows);
    // down: the CTAs a tile (they run together, so a cluster has to fit) whose waves take least, a wave's start and
    // sum counted as six stages.  Microseconds of the whole call by 2, 4 and 8: 8192 rows, 6144 x 6144, rank 64 70, 65, 73;
    // 4096 rows 47, 41, 45; 3000 rows 42, 35, 33; 16000 rows, 2048 x 6144, rank 32 89, 92, 99.
    a.ksteps = (p.K + 63) / 64;
    a.splits = 1;
    long long best = 0;
    for (int s = 1; s <= 8 && (s == 1 || s <= a.ksteps); s *= 2) {
        const int fit = down_clusters<T>(s);
        if (fit <= 0) continue;
        const long long cost = (tiles + fit - 1) / fit * ((a.ksteps + s - 1) / s + 6);
        if (!best || cost < best) {
            best = cost;
            a.splits = s;
        }
    }
    a.stage_bytes = kXBytes + a.r16 * 128;
    const int sums = (kTileRows * (p.R + 4) * 4 + 1023) / 1024 * 1024;
    a.stages = std::max((sums + a.stage_bytes - 1) / a.stage_bytes,
                        std::min(kMaxTileStages, (kHalfSm - 1024 - (int)sizeof(TileCtrl)) / a.stage_bytes));
    TileMaps m;
    cudaError_t e = cudaSuccess;
    const auto both = [&](CUtensorMap (&map)[2], const void *from, long long cols, long long ld, long long n) {
        if (e == cudaSuccess) e = rows_map(&map[0], from, 16, cols, ld, n, kTileRows);
        if (e == cudaSuccess) e = rows_map(&map[1], from, 16, cols, ld, n, kShortRows);
    };
    both(m.a, p.x, p.K, p.ldx, p.T);
    if (e == cudaSuccess) e = rows_map(&m.b, p.down, 16, p.K, p.K, (long long)p.A * p.R, a.r16);
    if (e != cudaSuccess) return e;
    e = launch_kernel(adapter_down_kernel<T>, dim3((unsigned)tiles * a.splits), dim3(kDownThreads),
                      1024 + (size_t)a.stages * a.stage_bytes + sizeof(TileCtrl), st, a.splits, a, m);
    if (e != cudaSuccess) return e;
    // up: the number of CTAs a tile whose waves take least, a CTA's start counted as three chunks
    a.chunks = (p.N + NC - 1) / NC;
    best = 0;
    for (int s = 1; s <= std::min(a.chunks, 32); ++s) {
        const long long cost = ((long long)tiles * s + slots - 1) / slots * ((a.chunks + s - 1) / s + 3);
        if (!best || cost < best) {
            best = cost;
            a.slices = s;
        }
    }
    a.stage_bytes = kXBytes + a.blocks * NC * 128;
    const int ubytes = a.parts * a.blocks * kXBytes;
    a.stages = std::min(kMaxTileStages, ((a.blocks == 1 ? 1 : 2) * kHalfSm - 1024 - (int)sizeof(TileCtrl) - ubytes) / a.stage_bytes);
    a.wide = (((uintptr_t)p.N * sizeof(Y)) | (uintptr_t)p.y) % 32 == 0;
    if (p.base) both(m.a, p.base, (long long)p.N * sizeof(Y) / 2, (long long)p.N * sizeof(Y) / 2, p.T);
    if (e == cudaSuccess) e = rows_map(&m.b, p.up, 16, p.R, p.R, (long long)p.A * p.N, NC);
    for (int i = 0; i < a.parts; ++i) both(m.u[i], a.u[i], a.r16, a.r16, rows);
    if (e != cudaSuccess) return e;
    return launch_kernel(adapter_up_kernel<T, Y>, dim3((unsigned)tiles * a.slices), dim3(kUpThreads),
                         1024 + (size_t)a.stages * a.stage_bytes + ubytes + sizeof(TileCtrl), st, 1, a, m);
}

// passes over as many rows as the workspace holds u for
template <typename T, typename Y>
cudaError_t launch_tiles(const AdapterArgs &p, int dtype, void *workspace, size_t workspace_bytes, cudaStream_t st)
{
    const long long cells = (p.T + kTileRows - 1) / kTileRows;
    const long long fit = (long long)((workspace_bytes - 256) / (row_bytes(p.R) * kTileRows));
    const long long each = std::min(cells, fit);
    char *ws = static_cast<char *>(workspace) + 256;
    for (long long c = 0; c < cells; c += each) {
        TileArgs a = {};
        a.p = p;
        a.cell0 = (int)c;
        a.cell1 = (int)std::min(cells, c + each);
        a.row0 = (int)c * kTileRows;
        const size_t part = (size_t)each * kTileRows * ((p.R + 15) / 16 * 16) * 2;
        a.parts = sizeof(Y) == 4 && dtype == MOE_DTYPE_BF16 ? 3 : 2;
        for (int i = 0; i < kMaxParts; ++i) a.u[i] = ws + i * part;
        a.back = reinterpret_cast<float *>(ws + kMaxParts * part);
        const cudaError_t e = launch_pass<T, Y>(a, dtype, st);
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

}  // namespace adapter
}  // namespace moe
