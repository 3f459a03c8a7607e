// mxfp4_gemm.cu -- launches of the MXFP4 products (kernel: gemm_tc.cuh) and their entry points.
#include <algorithm>

#include "gemm_tc.cuh"
#include "tensor_map.cuh"

namespace moe {

namespace {

using namespace gemm;

// e2m1 x e2m1 with ue8m0 scales, fp32 sums, both operands reduction-major, 128 lanes
constexpr uint32_t kIdescMx = (1u << 7) | (1u << 10) | (1u << 23) | ((uint32_t)(kM >> 4) << 24);

cudaError_t code_maps(Maps &m, const uint8_t *a0, const uint8_t *a1, long long arows, const uint8_t *b, int rows, int K,
                      int widest)
{
    cudaError_t e = rows_map(&m.a[0], a0, 8, K / 2, K / 2, arows, kM);
    if (e == cudaSuccess && a1) e = rows_map(&m.a[1], a1, 8, K / 2, K / 2, arows, kM);
    for (int k = 0; 16 * (k + 1) <= widest && e == cudaSuccess; ++k)
        e = rows_map(&m.b[k], b, 8, K / 2, K / 2, rows, 16 * (k + 1));
    return e;
}

// Few rows a group take tiles of 32 columns: more stages in flight, and a cluster a tile while
// tiles are fewer than SMs.
bool few_rows(int rows, int E) { return rows <= 24 * std::min(E, rows); }
constexpr int kFew = 32, kMany = 192;

template <Mode MODE, bool WHOLE>
cudaError_t run_as(Args &a, const Maps &m, cudaStream_t st)
{
    const int sms = num_sms();
    const int mtiles = (a.M + kM - 1) / kM, used = std::min(a.E, a.rows);
    const int widest = few_rows(a.rows, a.E) ? kFew : kMany;
    a.split = widest == kFew ? choose_split<MODE, kFew, WHOLE>((long long)mtiles * used, a.ksteps) : 1;
    a.width = a.split > 1 ? kSplitCols : widest;
    // at most this many tiles: every group's last chunk may be short
    const long long tiles = (long long)mtiles * std::min<long long>(a.rows, (a.rows + a.width - 1) / a.width + used);
    if (widest == kFew)
        return launch<MODE, kFew, WHOLE>(a, m, (int)std::min<long long>(tiles, 2 * sms / a.split) * a.split, st);
    return launch<MODE, kMany, WHOLE>(a, m, (int)std::min<long long>(tiles, sms), st);
}

template <Mode MODE>
cudaError_t run(Args &a, const Maps &m, cudaStream_t st)
{
    return a.sf_ld % 16 ? run_as<MODE, false>(a, m, st) : run_as<MODE, true>(a, m, st);
}

}  // namespace

cudaError_t launch_mxfp4_matmul(const uint8_t *x, const uint8_t *xs, int rows, const uint8_t *w, const uint8_t *ws,
                                int E, const int32_t *offsets, int N, int K, void *y, int dtype, int early, int32_t *err,
                                cudaStream_t st)
{
    Maps m;
    const cudaError_t e = code_maps(m, w, nullptr, (long long)E * N, x, rows, K, few_rows(rows, E) ? kFew : kMany);
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
    return run<kMxMul>(a, m, st);
}

cudaError_t launch_mxfp4_gate_up(const uint8_t *x, const uint8_t *xs, int rows, const uint8_t *wg, const uint8_t *sg,
                                 const uint8_t *wu, const uint8_t *su, int E, const int32_t *offsets, int F, int K,
                                 uint8_t *codes, uint8_t *scales, int early, int32_t *err,
                                 cudaStream_t st)
{
    Maps m;
    const cudaError_t e = code_maps(m, wg, wu, (long long)E * F, x, rows, K, few_rows(rows, E) ? kFew : kMany);
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
    return run<kMxGate>(a, m, st);
}

}  // namespace moe
