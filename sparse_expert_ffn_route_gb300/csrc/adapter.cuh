// adapter.cuh -- what the two kernels of the adapters (adapter.cu, adapter_tiles.cuh) share: arguments, and
// the tiles of a batch cut into segments.
#pragma once

#include "cluster_wait.cuh"
#include "launch.cuh"
#include "moe_internal.cuh"
#include "vec8.cuh"

namespace moe {
namespace adapter {

constexpr int kMaxRank = 128, kMaxAdapterDim = 65536, kMaxAdapters = 1 << 16, kMaxSegments = 1 << 20;
struct AdapterArgs {
    const void *x;
    long long ldx;
    const void *down, *up;
    const float *scale;
    const int32_t *offsets, *ids;
    const void *base;
    void *y;
    int T, S, K, N, R, A;
    int32_t *err;
};

// Tiles of `rows` rows on a fixed grid over the batch, cut by the segments: the part of grid cell c that is
// segment s's is tile c + s.  (A later part has a later cell or a later segment, so no two share a number.)
// In a list whose offsets are not in order the search may miss a segment, whose tiles are then left out; a tile that is
// found is a part of one segment within the rows, and no part has two numbers.
struct Tile {
    int lo, hi;      // rows; empty where the number is not used
    int adapter;     // -1: none
    bool bad;        // not an adapter: the rows become NaN
};

// by one warp
__device__ __forceinline__ Tile find_tile(const AdapterArgs &p, int tile, int rows, int lane)
{
    Tile t = {0, 0, -1, false};
    int s = 0, n = p.S;      // the last segment whose first tile is `tile` or before it lies in [s, s + n)
    while (n > 1) {
        const int step = (n + 31) / 32, at = lane * step;
        const bool before = at < n && p.offsets[s + at] / rows + s + at <= tile;
        const int got = __popc(__ballot_sync(0xffffffffu, before));
        if (got == 0) return t;
        n = min(step, n - (got - 1) * step);
        s += (got - 1) * step;
    }
    const int cell = tile - s, from = p.offsets[s], to = p.offsets[s + 1];
    if (cell < 0 || from < 0 || from > to || to > p.T) return t;
    t.lo = max(from, cell * rows);
    t.hi = (int)min((long long)to, ((long long)cell + 1) * rows);
    t.adapter = p.ids[s];
    t.bad = t.adapter < -1 || t.adapter >= p.A;
    return t;
}

// what is wrong with segment s, recorded
__device__ __forceinline__ void check_segment(const AdapterArgs &p, int s)
{
    const int from = p.offsets[s], to = p.offsets[s + 1], id = p.ids[s];
    if (from < 0 || from > to || to > p.T) atomicOr(p.err, kErrBadOffsets);
    if (id < -1 || id >= p.A) atomicOr(p.err, kErrBadAdapter);
}

// y = base (or zero, or NaN for a segment whose id is no adapter) for the tile's columns [n0, n1), by `threads` threads;
// rows and columns are whole 16-byte pieces, four of a thread on their way at once
template <typename Y>
__device__ __forceinline__ void pass_through(const AdapterArgs &p, const Tile &t, int n0, int n1, int tid, int threads)
{
    if (!t.bad && p.base == p.y) return;
    constexpr int N = 16 / sizeof(Y);
    union Piece {
        uint4 w;
        Y y[N];
        __device__ Piece() {}
    } fill;
#pragma unroll
    for (int j = 0; j < N; ++j) from_f32(fill.y[j], t.bad ? __int_as_float(0x7fc00000) : 0.0f);
    const bool copy = !t.bad && p.base;
    const int width = (n1 - n0) / N;
    const int total = (t.hi - t.lo) * width;   // (at most 128 rows of 2^14 pieces)
    for (int i0 = tid; i0 < total; i0 += 4 * threads) {
        uint4 v[4];
        size_t at[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int i = i0 + j * threads;
            if (i >= total) continue;
            const int row = i / width;
            at[j] = (size_t)(t.lo + row) * p.N + n0 + (i - row * width) * N;
            v[j] = copy ? *reinterpret_cast<const uint4 *>(static_cast<const Y *>(p.base) + at[j]) : fill.w;
        }
#pragma unroll
        for (int j = 0; j < 4; ++j)
            if (i0 + j * threads < total) *reinterpret_cast<uint4 *>(static_cast<Y *>(p.y) + at[j]) = v[j];
    }
}

}  // namespace adapter
}  // namespace moe
