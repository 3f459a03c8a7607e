// adapter_tiles.cuh -- adapters on tiles of 128 rows of one segment: both products on tcgen05, in one kernel.
//
// A cluster of 4 or 8 CTAs takes a tile.  Each CTA
//   1. sums u = x down^T (128 rows on the accumulator's lanes, the rank in its columns) over its share of the
//      inputs, fed by TMA;
//   2. adds its share of the rows' numbers over the cluster in rank order, through distributed shared memory,
//      and hands them to every CTA as the next product's operand;
//   3. forms u up^T for its share of the outputs and adds it to base: a thread of the epilogue holds 64
//      consecutive bytes of a row, which it reads ahead of the product.
// u goes through two 16-bit numbers a value, a high and a low part with the row's largest number brought to
// 2^13 (so that fp16 neither overflows nor loses the low part to its smallest numbers): 2^-17 of the row's
// largest and less is lost, and the product is formed twice, which costs nothing beside the memory.
//
// What it moves is x once and base and y once: bound by memory.  Two CTAs stand on an SM (half of its shared
// memory and of its TMEM each), so that one's first product, bound by its loads, runs beside another's
// outputs.
//
// Warps: 0 loads x and then up, 1 loads down, 2 issues the MMAs, 4-11 are the epilogue.  Every wait is bounded
// (cluster_wait.cuh); every thread goes to every cluster barrier.
#pragma once

#include <algorithm>

#include "adapter.cuh"
#include "gemm_tc.cuh"
#include "tensor_map.cuh"

namespace moe {
namespace adapter {

using gemm::expect_tx;
using gemm::tma_2d;
using gemm::uniform;

constexpr int kTileRows = 128;
constexpr int kTileThreads = 384;
constexpr int kEpiWarps = 8, kFirstEpi = 4;
constexpr int kMaxTileStages = 8;
constexpr int kXBytes = kTileRows * 128;
constexpr int kTmemCols = 256, kUpCol = 128, kUpStep = 64;   // u; then two buffers of outputs

struct TileArgs {
    AdapterArgs p;
    int ctas;            // of a cluster
    int r16;             // rank in steps of 16
    int blocks;          // of 64 ranks
    int ksteps;          // stages of 64 inputs in all
    int stages, stage_bytes, u_bytes;
    int chunks;          // of the outputs' columns
    int wide;            // base and y rows lie on 32-byte boundaries
    uint32_t idesc;      // without N
};

struct TileMaps {
    CUtensorMap x, down, up;
};

struct TileCtrl {
    uint64_t full[kMaxTileStages], empty[kMaxTileStages], ufull, dfull[2], dempty[2], fin;
    uint32_t tmem;
    int abort;
    Tile tile;
    float back[kTileRows];   // what undoes a row's scaling
};

__device__ __forceinline__ float4 ld_cluster_v4(uint32_t addr)
{
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

__device__ __forceinline__ void st_cluster_v2(uint32_t addr, uint2 v)
{
    asm volatile("st.shared::cluster.v2.b32 [%0], {%1, %2};" ::"r"(addr), "r"(v.x), "r"(v.y) : "memory");
}

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

__device__ __forceinline__ void fence_proxy_async_all() { asm volatile("fence.proxy.async;" ::: "memory"); }

// 64 consecutive bytes of a row, those of its first `n` 16-byte pieces; 32 at a time where rows allow it
__device__ __forceinline__ void load64(const char *p, uint32_t (&w)[16], int n, bool wide)
{
#pragma unroll
    for (int i = 0; i < 4; i += 2) {
        if (wide && i + 1 < n) {
            asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                         : "=r"(w[4 * i]), "=r"(w[4 * i + 1]), "=r"(w[4 * i + 2]), "=r"(w[4 * i + 3]), "=r"(w[4 * i + 4]),
                           "=r"(w[4 * i + 5]), "=r"(w[4 * i + 6]), "=r"(w[4 * i + 7])
                         : "l"(p + 16 * i)
                         : "memory");
        } else {
#pragma unroll
            for (int j = i; j < i + 2; ++j)
                if (j < n) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(p + 16 * j);
                    w[4 * j] = v.x;
                    w[4 * j + 1] = v.y;
                    w[4 * j + 2] = v.z;
                    w[4 * j + 3] = v.w;
                }
        }
    }
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

// had + scale * v of consecutive columns, in place
template <typename Y>
__device__ __forceinline__ void add_columns(uint32_t (&w)[sizeof(Y) * 4], const uint32_t (&v)[16], float scale)
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
        for (int j = 0; j < N; ++j) from_f32(u.y[j], fmaf(scale, __uint_as_float(v[i * N + j]), to_f32(u.y[j])));
        w[i] = u.w;
    }
}

template <typename T, typename Y>
__global__ void __launch_bounds__(kTileThreads, 2) adapter_tiles_kernel(const __grid_constant__ TileArgs a, const __grid_constant__ TileMaps maps)
{
    constexpr int CW = 64 / sizeof(Y);   // columns of a thread
    constexpr int NC = 2 * CW;           // of a chunk
    extern __shared__ __align__(1024) uint8_t smem_raw[];
    uint8_t *ring = reinterpret_cast<uint8_t *>(((uintptr_t)smem_raw + 1023) & ~(uintptr_t)1023);
    uint8_t *ubuf = ring + a.stages * a.stage_bytes;   // the rows' sums (fp32), then the operand
    TileCtrl *c = reinterpret_cast<TileCtrl *>(ubuf + a.u_bytes);
    const AdapterArgs &p = a.p;
    const int tid = threadIdx.x, lane = tid & 31, warp = uniform(tid >> 5);
    const int rank = blockIdx.x % a.ctas, number = blockIdx.x / a.ctas;
    if (tid < 32) {
        if (tid < kMaxTileStages) {
            mbar_init(&c->full[tid], 1);
            mbar_init(&c->empty[tid], 1);
        } else if (tid < kMaxTileStages + 2) {
            mbar_init(&c->dfull[tid - kMaxTileStages], 1);
            mbar_init(&c->dempty[tid - kMaxTileStages], kEpiWarps);
        } else if (tid == 31) {
            mbar_init(&c->ufull, 1);
            mbar_init(&c->fin, 1);
            c->abort = 0;
        }
        fence_mbar_init();
        __syncwarp();
    }
    // (at most two CTAs that want 256 columns fit an SM's shared memory, so that nobody holds what a CTA of
    // this cluster waits for while it waits for that CTA)
    if (warp == 2) gemm::tmem_alloc<false>(&c->tmem, kTmemCols);
    tc::fence_before_sync();
    __syncthreads();
    tc::fence_after_sync();
    pdl_wait();
    pdl_launch_dependents();
    if (warp == 0) {
        const Tile t = find_tile(p, number, kTileRows, lane);
        if (lane == 0) {
            c->tile = t;
            if (rank == 0 && number < p.S) check_segment(p, number);
        }
    }
    __syncthreads();
    const uint32_t tmem = uniform(c->tmem);
    const Tile t = c->tile;
    const int per = (a.chunks + a.ctas - 1) / a.ctas;
    const int chunk0 = min(a.chunks, rank * per), chunk1 = min(a.chunks, chunk0 + per);
    if (t.lo >= t.hi || t.adapter < 0 || t.bad) {   // (the same for the whole cluster)
        const int n0 = chunk0 * NC, n1 = min(p.N, chunk1 * NC);
        if (t.bad || p.base != p.y)
            for (int m = t.lo + warp; m < t.hi; m += kTileThreads / 32)
                for (int n = n0 + lane; n < n1; n += 32) {
                    const size_t at = (size_t)m * p.N + n;
                    Y v;
                    if (t.bad) from_f32(v, __int_as_float(0x7fc00000));
                    else if (p.base) v = static_cast<const Y *>(p.base)[at];
                    else from_f32(v, 0.0f);
                    static_cast<Y *>(p.y)[at] = v;
                }
        __syncthreads();
        if (warp == 2) gemm::tmem_dealloc<false>(tmem, kTmemCols);
        return;
    }
    const int kper = (a.ksteps + a.ctas - 1) / a.ctas;
    const int k0 = min(a.ksteps, rank * kper), ksteps = min(a.ksteps, k0 + kper) - k0, nchunks = chunk1 - chunk0;
    const uint32_t r0 = smem_u32(ring);
    const int adapter = uniform(t.adapter), row0 = uniform(t.lo);
    const auto wait = [&](uint64_t *bar, uint32_t parity) { return wait_or_abort(bar, parity, &c->abort, p.err); };

    // ---------------- u over this CTA's inputs -----------------------------------------------
    uint32_t it = 0, s = 0, phase = 0;   // stage of the ring, and its turn: x and down, then up
    bool ok = true;
    const auto next = [&] {
        ++it;
        if (++s == (uint32_t)a.stages) {
            s = 0;
            phase ^= 1;
        }
    };
    int loaded = 0;   // chunks of up
    const auto load_up = [&](int limit) {
        for (; loaded < limit && ok; ++loaded, next()) {
            if (it >= (uint32_t)a.stages && !(ok = wait(&c->empty[s], phase ^ 1))) break;
            const uint32_t bar = smem_u32(&c->full[s]);
            expect_tx(bar, a.blocks * NC * 128);
            for (int b = 0; b < a.blocks; ++b)
                tma_2d(r0 + s * a.stage_bytes + b * NC * 128, &maps.up, 64 * b, adapter * p.N + (chunk0 + loaded) * NC, bar);
        }
    };
    if (warp <= 1) {
        for (int k = 0; k < ksteps; ++k, next()) {
            if (it >= (uint32_t)a.stages && !(ok = wait(&c->empty[s], phase ^ 1))) break;
            const uint32_t bar = smem_u32(&c->full[s]), to = r0 + s * a.stage_bytes;
            if (warp == 0) {
                expect_tx(bar, kXBytes + a.r16 * 128);
                tma_2d(to, &maps.x, 64 * (k0 + k), row0, bar);
            } else {
                tma_2d(to + kXBytes, &maps.down, 64 * (k0 + k), adapter * p.R, bar);
            }
        }
        if (warp == 0) load_up(min(nchunks, a.stages));   // on their way during the exchange
    } else if (warp == 2) {
        const uint32_t idesc = a.idesc | (uint32_t)(a.r16 >> 3) << 17;
        for (int k = 0; k < ksteps; ++k, next()) {
            if (!(ok = wait(&c->full[s], phase))) break;
            tc::fence_after_sync();
            const uint64_t xd = tc::sdesc_kmajor_sw128(r0 + s * a.stage_bytes), dd = tc::sdesc_kmajor_sw128(r0 + s * a.stage_bytes + kXBytes);
#pragma unroll
            for (int j = 0; j < 4; ++j) gemm::mma_f16(tmem, xd + 2 * j, dd + 2 * j, idesc, k > 0 || j > 0);
            tc::commit_elect(&c->empty[s]);
        }
        tc::commit_elect(&c->ufull);
    } else if (warp >= kFirstEpi) {
        const int row = (warp & 3) * 32 + lane;
        float *to = reinterpret_cast<float *>(ubuf) + row * (p.R + 4);
        if (ksteps > 0) {
            ok = wait(&c->ufull, 0);
            tc::fence_after_sync();
        }
        for (int r = 16 * ((warp - kFirstEpi) >> 2); r < a.r16; r += 32) {
            uint32_t v[16];
            if (ksteps > 0) {
                tc::ld16(tmem + ((uint32_t)((warp & 3) * 32) << 16) + r, v);
                tc::wait_ld();
#pragma unroll
                for (int i = 0; i < 16; ++i) asm volatile("" : "+r"(v[i]));   // read after the wait
            } else {
#pragma unroll
                for (int i = 0; i < 16; ++i) v[i] = 0;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 4)
                if (r + i < p.R) *reinterpret_cast<uint4 *>(to + r + i) = make_uint4(v[i], v[i + 1], v[i + 2], v[i + 3]);
        }
        tc::fence_before_sync();
    }
    __syncwarp();
    cluster_sync();   // every CTA's sums are there

    // ---------------- added over the cluster, and cut into two 16-bit parts ---------------------
    constexpr int kMost = kTileRows / 4 / kEpiWarps;   // rows of a warp
    const int rows = kTileRows / a.ctas;
    uint2 hi[kMost], lo[kMost];
    float back[kMost];
    if (warp >= kFirstEpi) {
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int mine = warp - kFirstEpi + i * kEpiWarps, row = rank * rows + mine;
            if (mine >= rows) continue;
            float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            if (4 * lane < p.R) {
                const uint32_t at = smem_u32(ubuf) + (uint32_t)(row * (p.R + 4) + 4 * lane) * 4;
                for (int q = 0; q < a.ctas; ++q) {
                    const float4 w = ld_cluster_v4(map_rank(at, q));
                    v[0] += w.x;
                    v[1] += w.y;
                    v[2] += w.z;
                    v[3] += w.w;
                }
            }
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
            back[i] = __uint_as_float((uint32_t)(127 - shift) << 23);
            union {
                uint2 w;
                T t[4];
            } h, l;
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                from_f32(h.t[j], v[j] * by);
                const float had = to_f32(h.t[j]), rest = v[j] * by - had;
                from_f32(l.t[j], fabsf(had) <= 3.4e38f ? rest : 0.0f);
            }
            hi[i] = h.w;
            lo[i] = l.w;
        }
    }
    __syncwarp();
    cluster_sync();   // the sums have been read
    if (warp >= kFirstEpi) {
#pragma unroll
        for (int i = 0; i < kMost; ++i) {
            const int mine = warp - kFirstEpi + i * kEpiWarps, row = rank * rows + mine;
            if (mine >= rows) continue;
            const int r = 4 * lane;
            const uint32_t at = smem_u32(ubuf) + (r >> 6) * kXBytes + row * 128 + ((((r & 63) >> 3) ^ (row & 7)) << 4) + (r & 4) * 2;
            for (int q = 0; q < a.ctas; ++q) {
                if (r < a.r16) {
                    const uint32_t to = map_rank(at, q);
                    st_cluster_v2(to, hi[i]);
                    st_cluster_v2(to + a.blocks * kXBytes, lo[i]);
                }
                if (lane == 0) st_cluster_f32(map_rank(smem_u32(&c->back[row]), q), back[i]);
            }
        }
    }
    fence_proxy_async_all();
    __syncwarp();
    cluster_sync();   // the operand is there

    // ---------------- this CTA's outputs -----------------------------------------------------
    if (warp == 0) {
        load_up(nchunks);
        // the last commits on `empty` land before this CTA's shared memory is another kernel's
        for (uint32_t j = it > (uint32_t)a.stages ? it - a.stages : 0; j < it && ok; ++j) ok = wait(&c->empty[j % a.stages], (j / a.stages) & 1);
    } else if (warp == 2) {
        fence_proxy_async_all();
        tc::fence_after_sync();
        const uint32_t idesc = a.idesc | (uint32_t)(NC >> 3) << 17, u0 = smem_u32(ubuf);
        for (int j = 0; j < nchunks && ok; ++j, next()) {
            const uint32_t buf = j & 1, use = j >> 1, d = tmem + kUpCol + buf * kUpStep;
            if (use >= 1 && !(ok = wait(&c->dempty[buf], (use - 1) & 1))) break;
            if (!(ok = wait(&c->full[s], phase))) break;
            tc::fence_after_sync();
            uint32_t first = 0;
            for (int part = 0; part < 2; ++part)
                for (int k = 0; k < a.r16; k += 16) {
                    const uint64_t ud = tc::sdesc_kmajor_sw128(u0 + (part * a.blocks + (k >> 6)) * kXBytes) + ((k & 63) >> 3);
                    const uint64_t wd = tc::sdesc_kmajor_sw128(r0 + s * a.stage_bytes + (k >> 6) * NC * 128) + ((k & 63) >> 3);
                    gemm::mma_f16(d, ud, wd, idesc, first);
                    first = 1;
                }
            tc::commit_elect(&c->empty[s]);
            tc::commit_elect(&c->dfull[buf]);
        }
        tc::commit_elect(&c->fin);
    } else if (warp >= kFirstEpi) {
        const int part = (warp - kFirstEpi) >> 2, local = (warp & 3) * 32 + lane, row = t.lo + local;
        const bool on = row < t.hi;
        const float scale = (p.scale ? p.scale[adapter] : 1.0f) * c->back[local];
        const uint32_t tl = tmem + ((uint32_t)((warp & 3) * 32) << 16) + kUpCol + part * CW;
        const size_t line = (size_t)row * p.N;
        uint32_t ahead[16];
        const auto pieces = [&](int j) { return min(4, (p.N - ((chunk0 + j) * NC + part * CW)) / (CW / 4)); };   // below 1: none
        const auto at = [&](int j) { return (line + (chunk0 + j) * NC + part * CW) * sizeof(Y); };
        const auto fetch = [&](int j) {
#pragma unroll
            for (int i = 0; i < 16; ++i) ahead[i] = 0;
            if (p.base && on && j < nchunks) load64(static_cast<const char *>(p.base) + at(j), ahead, pieces(j), a.wide);
        };
        fetch(0);
        for (int j = 0; j < nchunks && ok; ++j) {
            const uint32_t buf = j & 1, use = j >> 1;
            uint32_t w[16];
#pragma unroll
            for (int i = 0; i < 16; ++i) w[i] = ahead[i];
            fetch(j + 1);
            if (!(ok = wait(&c->dfull[buf], use & 1))) break;
            tc::fence_after_sync();
            __syncwarp();
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
                add_columns<Y>(*reinterpret_cast<uint32_t(*)[W]>(&w[h / 16 * W]), v, scale);
            }
            if (on) store64(static_cast<char *>(p.y) + at(j), w, pieces(j), a.wide);
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
    cluster_sync();   // (a CTA that gives up writes to the others' memory)
}

template <typename T, typename Y>
cudaError_t launch_tiles(const AdapterArgs &p, int dtype, cudaStream_t st)
{
    constexpr int NC = 128 / sizeof(Y);
    TileArgs a = {};
    a.p = p;
    const int tiles = (int)((p.T + kTileRows - 1) / kTileRows) + p.S;
    a.ctas = 4 * tiles >= 2 * num_sms() ? 4 : 8;
    a.r16 = (p.R + 15) / 16 * 16;
    a.blocks = (p.R + 63) / 64;
    a.ksteps = (p.K + 63) / 64;
    a.chunks = (p.N + NC - 1) / NC;
    a.stage_bytes = kXBytes + a.r16 * 128;
    a.u_bytes = (std::max(2 * a.blocks * kXBytes, kTileRows * (p.R + 4) * 4) + 1023) / 1024 * 1024;
    // half of an SM's shared memory up to a rank of 64
    const int budget = (a.blocks == 1 ? 112 : 224) * 1024 - 1024 - (int)sizeof(TileCtrl) - a.u_bytes;
    a.stages = std::min(kMaxTileStages, budget / a.stage_bytes);
    const uint32_t f = dtype == MOE_DTYPE_BF16 ? 1u : 0u;
    a.idesc = (1u << 4) | (f << 7) | (f << 10) | ((uint32_t)(kTileRows >> 4) << 24);
    const uintptr_t bits = (uintptr_t)p.N * sizeof(Y) | (uintptr_t)p.y | (uintptr_t)p.base;
    a.wide = bits % 32 == 0;
    TileMaps m;
    cudaError_t e = rows_map(&m.x, p.x, 16, p.K, p.ldx, p.T, kTileRows);
    if (e == cudaSuccess) e = rows_map(&m.down, p.down, 16, p.K, p.K, (long long)p.A * p.R, a.r16);
    if (e == cudaSuccess) e = rows_map(&m.up, p.up, 16, p.R, p.R, (long long)p.A * p.N, NC);
    if (e != cudaSuccess) return e;
    const size_t smem = 1024 + (size_t)a.stages * a.stage_bytes + a.u_bytes + sizeof(TileCtrl);
    return launch_kernel(adapter_tiles_kernel<T, Y>, dim3((unsigned)tiles * a.ctas), dim3(kTileThreads), smem, st, a.ctas, a, m);
}

}  // namespace adapter
}  // namespace moe
