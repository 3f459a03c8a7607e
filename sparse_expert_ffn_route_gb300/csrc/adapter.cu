// adapter.cu -- low-rank adapters of many requests beside a projection they share:
//   y[p] = base[p] + scale[a] (x[p] down[a]^T) up[a]^T,  a = ids[s], for the rows p of segment s.
//
// Many rows a segment: tiles of 128 rows on the tensor cores (adapter_tiles.cuh).
//
// Few rows a segment (a decode batch).  A cluster of 8 CTAs takes up to 4 rows of one segment: each CTA forms the
// rows' R numbers over its eighth of the inputs and sends them to all eight, which add them in rank order, and
// each writes its eighth of the outputs.  One launch, nothing goes through global memory in between.  It is a
// chain of waits (list, weights, cluster, outputs), so what can be asked for early is: a thread's first row of up
// comes during the first product, and the sums are pushed into the others' shared memory, not fetched from there
// (64 tokens of 32 adapters, 6144 x 2048, rank 16: 10.1 us with the sums fetched and x staged, 6.9 like this).
#include <algorithm>
#include <cmath>

#include "adapter_tiles.cuh"

namespace moe {

using namespace adapter;

namespace {

constexpr int kFewRows = 4;       // rows of a tile
constexpr int kFewCluster = 8;
constexpr int kFewThreads = 256;

__device__ __forceinline__ void st_cluster_f32(uint32_t addr, float v)
{
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(addr), "f"(v) : "memory");
}

// Sums over this CTA's inputs k of x[m][k] down[r][k], M rows, two r of a warp at a time, sent to every CTA of the
// cluster: to[rank][m][r].
template <typename T, int M>
__device__ __forceinline__ void few_down(const T *x, long long ldx, int rows, int width, const T *down, long long ldd, int R,
                                         float *to, int rank, int warp, int lane)
{
    constexpr int U = 2, V = U * M;   // V: a power of two, at most 16
    bool started = false;
    for (int r0 = warp * U; r0 < R; r0 += kFewThreads / 32 * U) {
        float acc[V];
#pragma unroll
        for (int i = 0; i < V; ++i) acc[i] = 0.0f;
#pragma unroll(M <= 2 ? 2 : 1)
        for (int k = lane * 8; k < width; k += 256) {
            float d[U][8], f[8];
            Vec8<T> v[U], w;
#pragma unroll
            for (int u = 0; u < U; ++u) v[u].load(down + (r0 + u) * ldd + k);
#pragma unroll
            for (int u = 0; u < U; ++u) v[u].get(d[u]);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                if (M > 2 && m >= rows) break;
                w.load(x + min(m, rows - 1) * ldx + k);
                w.get(f);
#pragma unroll
                for (int u = 0; u < U; ++u)
#pragma unroll
                    for (int i = 0; i < 8; ++i) acc[u * M + m] = fmaf(f[i], d[u][i], acc[u * M + m]);
            }
        }
        ReduceScatter<V, 16>::run(acc, lane);
        constexpr int each = 32 / V;       // lanes that hold one value
        const int i = lane / each;
        if (!started) gemm::cluster_wait();    // every CTA of the cluster runs
        started = true;
        const uint32_t at = smem_u32(to + (rank * kFewRows + i % M) * kMaxRank + r0 + i / M);
        for (int q = lane % each; q < kFewCluster; q += each) st_cluster_f32(map_rank(at, q), acc[0]);
        __syncwarp();
    }
    if (!started) gemm::cluster_wait();
}

template <typename T, typename Y, int M>
__device__ __forceinline__ void few_up(const AdapterArgs &p, const Tile &t, const float *u, const T *up, float scale, int n0, int n1,
                                       const Vec8<T> (&ahead)[2])
{
    const int rows = t.hi - t.lo;
    for (int n = n0 + threadIdx.x; n < n1; n += kFewThreads) {
        float acc[M];
#pragma unroll
        for (int m = 0; m < M; ++m) acc[m] = 0.0f;
        const T *b = up + (size_t)n * p.R;
        const bool first = n < n0 + kFewThreads;
        const auto add = [&](const Vec8<T> &v, int r) {
            float f[8], g[8];
            v.get(f);
#pragma unroll
            for (int m = 0; m < M; ++m) {
                Vec8<float> w;
                w.load(u + m * kMaxRank + r);
                w.get(g);
#pragma unroll
                for (int i = 0; i < 8; ++i) acc[m] = fmaf(g[i], f[i], acc[m]);
            }
        };
        int r = 0;
        if (first) {
            add(ahead[0], 0);
            if (p.R > 8) add(ahead[1], 8);
            r = 16;
        }
        for (; r < p.R; r += 8) {
            Vec8<T> v;
            v.load(b + r);
            add(v, r);
        }
#pragma unroll
        for (int m = 0; m < M; ++m)
            if (m < rows) {
                const size_t at = (size_t)(t.lo + m) * p.N + n;
                const float had = p.base ? to_f32(static_cast<const Y *>(p.base)[at]) : 0.0f;
                from_f32(static_cast<Y *>(p.y)[at], fmaf(scale, acc[m], had));
            }
    }
}

template <typename T, typename Y>
__global__ void __launch_bounds__(kFewThreads, 4) adapter_few_kernel(const AdapterArgs p)
{
    __shared__ __align__(16) float s_part[kFewCluster * kFewRows * kMaxRank], s_u[kFewRows * kMaxRank];
    pdl_wait();
    pdl_launch_dependents();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int tile = blockIdx.x / kFewCluster, rank = blockIdx.x % kFewCluster;
    const Tile t = find_tile(p, tile, kFewRows, lane);   // (by every warp, for want of a barrier)
    if (warp == 0 && lane == 0 && rank == 0 && tile < p.S) check_segment(p, tile);
    const int rows = t.hi - t.lo;
    if (rows <= 0) return;                       // (the same for the whole cluster)
    const int nslice = (p.N / 8 + kFewCluster - 1) / kFewCluster * 8;
    const int n0 = min(p.N, rank * nslice), n1 = min(p.N, n0 + nslice);
    if (t.adapter < 0 || t.bad) return pass_through<Y>(p, t, n0, n1, tid, kFewThreads);
    gemm::cluster_arrive();
    // this thread's first row of up, on its way during the first product
    const T *up = static_cast<const T *>(p.up) + (size_t)t.adapter * p.N * p.R;
    Vec8<T> ahead[2];
    ahead[0].zero();
    ahead[1].zero();
    if (n0 + tid < n1) {
        ahead[0].load(up + (size_t)(n0 + tid) * p.R);
        if (p.R > 8) ahead[1].load(up + (size_t)(n0 + tid) * p.R + 8);
    }
    const float scale = p.scale ? p.scale[t.adapter] : 1.0f;
    const int kslice = (p.K / 8 + kFewCluster - 1) / kFewCluster * 8;
    const int k0 = min(p.K, rank * kslice), width = min(p.K, k0 + kslice) - k0;
    const int m_up = rows == 1 ? 1 : rows == 2 ? 2 : 4;
    const T *x = static_cast<const T *>(p.x) + (size_t)t.lo * p.ldx + k0;
    const T *down = static_cast<const T *>(p.down) + (size_t)t.adapter * p.R * p.K + k0;
    switch (m_up) {
    case 1: few_down<T, 1>(x, p.ldx, rows, width, down, p.K, p.R, s_part, rank, warp, lane); break;
    case 2: few_down<T, 2>(x, p.ldx, rows, width, down, p.K, p.R, s_part, rank, warp, lane); break;
    default: few_down<T, 4>(x, p.ldx, rows, width, down, p.K, p.R, s_part, rank, warp, lane); break;
    }
    __syncwarp();
    cluster_sync();                              // every CTA's sums are there, and nothing is sent after this
    for (int i = tid; i < m_up * p.R; i += kFewThreads) {
        const int at = i / p.R * kMaxRank + i % p.R;
        float sum = 0.0f;
#pragma unroll
        for (int c = 0; c < kFewCluster; ++c) sum += s_part[c * kFewRows * kMaxRank + at];
        s_u[at] = sum;
    }
    __syncthreads();
    switch (m_up) {
    case 1: few_up<T, Y, 1>(p, t, s_u, up, scale, n0, n1, ahead); break;
    case 2: few_up<T, Y, 2>(p, t, s_u, up, scale, n0, n1, ahead); break;
    default: few_up<T, Y, 4>(p, t, s_u, up, scale, n0, n1, ahead); break;
    }
}

// f(T()) of the two 16-bit types
template <typename F>
auto with_half(int dtype, F &&f)
{
    return dtype == MOE_DTYPE_BF16 ? f(__nv_bfloat16()) : f(__half());
}

cudaError_t launch_few(const AdapterArgs &p, int dtype, int y_dtype, cudaStream_t st)
{
    const long long tiles = (p.T + kFewRows - 1) / kFewRows + p.S;
    return with_half(dtype, [&](auto t) {
        return with_dtype(y_dtype, [&](auto y) {
            return launch_kernel(adapter_few_kernel<decltype(t), decltype(y)>, dim3((unsigned)(tiles * kFewCluster)), dim3(kFewThreads),
                                 0, st, kFewCluster, p);
        });
    });
}

// Which kernels, by what they take on GB300 in microseconds.  The clusters' time goes with their number for each SM
// and with a tile's products; a tile of 128 rows costs its copies whatever stands in it.  Measured, clusters and tiles
// (rows, segments, K, N, rank): 1, 1, 2048, 6144, 16: 4.8, 6.9; 1, 1, 6144, 6144, 64: 10.3, 8.6; 64, 64, 6144, 2048, 16: 7.1,
// 17.2; 64, 64, 6144, 6144, 64: 25.7, 31.8; 64, 16, 6144, 6144, 64: 24.9, 13.6; 128, 16, 6144, 2048, 16: 8.9, 10.6; 256, 64,
// 6144, 2048, 16: 14.8, 16.9; 256, 64, 6144, 6144, 64: 58.1, 30.5; 256, 256, 6144, 6144, 16: 27.2, 86.1.  An fp32 y
// costs the tiles more columns' chunks, and with bf16 operands a third part of u, the clusters nothing (bf16, fp32 y): 1, 1, 6144,
// 6144, 64: 9.7, 11.2; 1, 1, 4096, 4096, 64: 7.5, 9.1; 1, 1, 6144, 6144, 128: 16.0, 13.3; 4, 1, 2048, 2048, 64: 8.8, 7.1.
bool few_rows(const AdapterArgs &p, int dtype, int y_dtype)
{
    const double each = std::max(1.0, (double)p.T / p.S), rows = std::min(each, (double)kFewRows);
    const double sms = p.S * std::ceil(each / kFewRows) * kFewCluster / num_sms(), work = (double)p.R * (p.K + p.N) / 1e5;
    const double few = 4 + 0.5 * sms + std::max(1.0, sms) * work * (0.45 + 0.35 * rows);
    const double wide = y_dtype == MOE_DTYPE_F32 ? 2.3e-4 + (dtype == MOE_DTYPE_BF16 ? 5e-5 + 2e-6 * p.R : 0) : 0;
    const double tiles = 6 + 2.1e-4 * (p.K + p.N) + wide * p.N + (p.S + (double)p.T / adapter::kTileRows) * (0.02 + 2.2e-5 * (p.K + p.N));
    return few < tiles;
}

cudaError_t launch_adapter(const AdapterArgs &p, int dtype, int y_dtype, void *workspace, size_t bytes, cudaStream_t st)
{
    if (few_rows(p, dtype, y_dtype)) return launch_few(p, dtype, y_dtype, st);
    return with_half(dtype, [&](auto t) {
        return with_dtype(y_dtype, [&](auto y) { return adapter::launch_tiles<decltype(t), decltype(y)>(p, dtype, workspace, bytes, st); });
    });
}

bool off(const void *p, size_t a) { return ((uintptr_t)p % a) != 0; }

int done(cudaError_t e, const char *what)
{
    if (e != cudaSuccess) return set_error(MOE_ERR_CUDA, "%s: %s", what, cudaGetErrorString(e));
    return set_error(MOE_OK, "%s", "");
}

}  // namespace

}  // namespace moe

using namespace moe;

#define ADAPTER_PTR(p, a)                                                                               \
    do {                                                                                                \
        if (!(p)) return set_error(MOE_ERR_ARG, "%s is NULL", #p);                                      \
        if (off((p), (a))) return set_error(MOE_ERR_ALIGN, "%s is not %d-byte aligned", #p, (int)(a));  \
    } while (0)

extern "C" {

size_t moe_adapter_workspace_size(int T, int rank)
{
    if (T < 0 || T > 1 << 24 || rank < 8 || rank > kMaxRank || rank % 8) return 0;
    return 256 + (size_t)(T + adapter::kTileRows - 1) / adapter::kTileRows * adapter::kTileRows * adapter::row_bytes(rank);
}

int moe_adapter_matmul(const void *x, long long ldx, int dtype, int T, int K, const void *down, const void *up, const float *scale,
                       int adapters, int rank, int N, const int32_t *offsets, const int32_t *ids, int segments, const void *base,
                       void *y, int y_dtype, void *workspace, size_t workspace_bytes, void *stream)
{
    int rc;
    if (dtype != MOE_DTYPE_BF16 && dtype != MOE_DTYPE_F16) return set_error(MOE_ERR_ARG, "dtype must be bf16 or fp16 (got %d)", dtype);
    if (y_dtype != MOE_DTYPE_F32 && y_dtype != MOE_DTYPE_BF16 && y_dtype != MOE_DTYPE_F16)
        return set_error(MOE_ERR_ARG, "unknown dtype %d", y_dtype);
    if (T < 0 || T > 1 << 24) return set_error(MOE_ERR_SHAPE, "T must be in [0, 2^24] (got %d)", T);
    if (K < 8 || K > kMaxAdapterDim || K % 8)
        return set_error(MOE_ERR_SHAPE, "K must be a multiple of 8 in [8, %d] (got %d)", kMaxAdapterDim, K);
    if (N < 8 || N > kMaxAdapterDim || N % 8)
        return set_error(MOE_ERR_SHAPE, "N must be a multiple of 8 in [8, %d] (got %d)", kMaxAdapterDim, N);
    if (rank < 8 || rank > kMaxRank || rank % 8)
        return set_error(MOE_ERR_SHAPE, "rank must be a multiple of 8 in [8, %d] (got %d)", kMaxRank, rank);
    if (adapters < 1 || adapters > kMaxAdapters) return set_error(MOE_ERR_SHAPE, "adapters must be in [1, 2^16] (got %d)", adapters);
    if ((long long)adapters * N > INT32_MAX) return set_error(MOE_ERR_SHAPE, "adapters * N must be below 2^31");
    if (segments < 1 || segments > kMaxSegments) return set_error(MOE_ERR_SHAPE, "segments must be in [1, 2^20] (got %d)", segments);
    if (ldx < K) return set_error(MOE_ERR_SHAPE, "ldx must be at least K (got %lld)", ldx);
    if (ldx % 8) return set_error(MOE_ERR_ALIGN, "rows of x are not 16-byte aligned (ldx %lld)", ldx);
    if (T == 0) return done(cudaSuccess, "");
    ADAPTER_PTR(x, 16);
    ADAPTER_PTR(down, 16);
    ADAPTER_PTR(up, 16);
    ADAPTER_PTR(offsets, 4);
    ADAPTER_PTR(ids, 4);
    ADAPTER_PTR(y, 16);
    if (off(base, 16)) return set_error(MOE_ERR_ALIGN, "base is not 16-byte aligned");
    if (off(scale, 4)) return set_error(MOE_ERR_ALIGN, "scale is not 4-byte aligned");
    if (!workspace) return set_error(MOE_ERR_WORKSPACE, "workspace is NULL");
    if (off(workspace, 256)) return set_error(MOE_ERR_ALIGN, "workspace is not 256-byte aligned");
    const size_t need = moe_adapter_workspace_size(std::min(T, adapter::kTileRows), rank);
    if (workspace_bytes < need) return set_error(MOE_ERR_WORKSPACE, "workspace has %zu bytes; %zu needed", workspace_bytes, need);
    if ((rc = require_device())) return rc;
    AdapterArgs p = {};
    p.x = x;
    p.ldx = ldx;
    p.down = down;
    p.up = up;
    p.scale = scale;
    p.offsets = offsets;
    p.ids = ids;
    p.base = base;
    p.y = y;
    p.T = T;
    p.S = segments;
    p.K = K;
    p.N = N;
    p.R = rank;
    p.A = adapters;
    p.err = static_cast<int32_t *>(workspace);
    return done(launch_adapter(p, dtype, y_dtype, workspace, workspace_bytes, (cudaStream_t)stream), "adapter launch");
}

}  // extern "C"
