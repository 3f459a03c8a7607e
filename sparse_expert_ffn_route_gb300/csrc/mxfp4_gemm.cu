// mxfp4_gemm.cu -- launches of the MXFP4 products (kernel: gemm_tc.cuh) and their entry points.
#include <algorithm>

#include "gemm_tc.cuh"
#include "tensor_map.cuh"

namespace moe {

namespace {

using namespace gemm;

// e2m1 x e2m1 with ue8m0 scales, fp32 sums, both operands reduction-major (without the lanes)
constexpr uint32_t kIdescMx = (1u << 7) | (1u << 10) | (1u << 23);

// Few rows a group take tiles of 32 columns on one SM: more stages in flight, two CTAs an SM, and
// a cluster a tile while tiles are fewer than SMs.  Microseconds of a product, few columns and many,
// by rows a group: 6144 x 6144 8: 8.8, 11.0; 24: 11.4, 11.1; 32 groups of 6144 x 2048 8: 38, 43;
// 24: 40, 44; 48: 55, 45.
bool few_rows(int rows, int E) { return rows <= 24 * std::min(E, rows); }
constexpr int kFew = 32, kMany = 224;

cudaError_t code_maps(Maps &m, const uint8_t *a0, const uint8_t *a1, long long arows, const uint8_t *b, int rows, int K,
                      bool few)
{
    cudaError_t e = rows_map(&m.a[0], a0, 8, K / 2, K / 2, arows, kM);
    if (e == cudaSuccess && a1) e = rows_map(&m.a[1], a1, 8, K / 2, K / 2, arows, kM);
    for (int k = 0; 16 * (k + 1) <= (few ? kFew : kMany / 2) && e == cudaSuccess; ++k)
        e = rows_map(&m.b[k], b, 8, K / 2, K / 2, rows, 16 * (k + 1));
    return e;
}

template <Mode MODE, bool WHOLE>
cudaError_t run_as(Args &a, const Maps &m, bool few, cudaStream_t st)
{
    const int sms = num_sms(), used = std::min(a.E, a.rows);
    // a bound on the tiles: every group's last chunk may be short
    const auto tiles = [&](int mtiles) {
        return (long long)mtiles * std::min<long long>(a.rows, (a.rows + a.width - 1) / a.width + used);
    };
    if (few) {
        const int mtiles = (a.M + kM - 1) / kM;
        a.idesc |= (uint32_t)(kM >> 4) << 24;
        a.split = choose_split<MODE, kFew, WHOLE>(mtiles * std::min<long long>(a.rows, a.rows / kSplitCols + used), a.ksteps);
        a.width = a.split > 1 ? kSplitCols : kFew;
        return launch<MODE, kFew, WHOLE>(a, m, (int)std::min<long long>(tiles(mtiles), 2 * sms / a.split) * a.split, st);
    }
    const int pairs = sms / 2;
    a.idesc |= (uint32_t)(2 * kM >> 4) << 24;
    a.split = 1;
    a.width = kMany;
    int lanes = 2 * kM;
    if (a.E == 1) {
        // One group: the tile whose waves of pairs take least.  A stage costs the pipe 2 cycles a
        // column and sum, or what L2 feeds: 50 bytes a cycle; a tile 1500 cycles more, and its epilogue
        // where its sums take both halves of TMEM.  A product may hold twice the weight rows: 46 KB
        // a stage for 896 cycles of the pipe in place of 33 KB for 448.
        double best = 0;
        for (int two = MODE == kMxGate; two < 2; ++two)
            for (int w = kMany; w >= 32; w -= 32) {
                const int na = two ? 2 : 1, l = MODE == kMxMul && two ? 4 * kM : 2 * kM;
                const long long t = (long long)((a.M + l - 1) / l) * ((a.rows + w - 1) / w);
                const double stage = std::max(2.0 * na * w, (16384.0 * na + 64.0 * w) / 50);
                const double cost = (double)((t + pairs - 1) / pairs) * (a.ksteps * stage + 1500 + (na * w > 224 ? 20.0 * w : 0.0));
                if (best == 0 || cost < best) {
                    best = cost;
                    a.width = w;
                    lanes = l;
                }
            }
    }
    const int grid = 2 * (int)std::min<long long>(tiles((a.M + lanes - 1) / lanes), pairs);
    if constexpr (MODE == kMxMul)
        if (lanes > 2 * kM) return launch<kMxMul2, kMany, WHOLE>(a, m, grid, st);
    return launch<MODE, kMany, WHOLE>(a, m, grid, st);
}

template <Mode MODE>
cudaError_t run(Args &a, const Maps &m, bool few, cudaStream_t st)
{
    return a.sf_ld % 16 ? run_as<MODE, false>(a, m, few, st) : run_as<MODE, true>(a, m, few, st);
}

}  // namespace

cudaError_t launch_mxfp4_matmul(const uint8_t *x, const uint8_t *xs, int rows, const uint8_t *w, const uint8_t *ws,
                                int E, const int32_t *offsets, int N, int K, void *y, int dtype, int early, int32_t *err,
                                cudaStream_t st)
{
    Maps m;
    const bool few = few_rows(rows, E);
    const cudaError_t e = code_maps(m, w, nullptr, (long long)E * N, x, rows, K, few);
    if (e != cudaSuccess) return e;
    Args a = {};
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.M = N;
    a.ksteps = (K + 255) / 256;
    a.sfa[0] = ws;
    a.sfb = xs;
    a.sf_ld = K / 32;
    a.sfa_rows = (long long)E * N;
    a.out[0] = y;
    a.ld = N;
    a.dtype = dtype;
    a.idesc = kIdescMx;
    a.early = early;
    a.err = err;
    return run<kMxMul>(a, m, few, st);
}

cudaError_t launch_mxfp4_gate_up(const uint8_t *x, const uint8_t *xs, int rows, const uint8_t *wg, const uint8_t *sg,
                                 const uint8_t *wu, const uint8_t *su, int E, const int32_t *offsets, int F, int K,
                                 uint8_t *codes, uint8_t *scales, int early, int32_t *err,
                                 cudaStream_t st)
{
    Maps m;
    const bool few = few_rows(rows, E);
    const cudaError_t e = code_maps(m, wg, wu, (long long)E * F, x, rows, K, few);
    if (e != cudaSuccess) return e;
    Args a = {};
    a.offsets = offsets;
    a.E = E;
    a.rows = rows;
    a.M = F;
    a.ksteps = (K + 255) / 256;
    a.sfa[0] = sg;
    a.sfa[1] = su;
    a.sfb = xs;
    a.sf_ld = K / 32;
    a.sfa_rows = (long long)E * F;
    a.out[0] = codes;
    a.out[1] = scales;
    a.ld = F;
    a.idesc = kIdescMx;
    a.early = early;
    a.err = err;
    return run<kMxGate>(a, m, few, st);
}

}  // namespace moe
