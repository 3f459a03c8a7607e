// selftest.cu -- exercises the error path of the library's bounded device-side waits without
// faulting or hanging the GPU.  A pair of CTAs waits on mbarriers that nothing arrives at: one warp
// gives up after a bounded number of polls and records kErrTimeout in the workspace error word, the
// other three, which go on waiting in short turns, end because it told them, the way the tensor-core
// kernels' warps do between tiles (cluster_wait.cuh).  The host reads the word with moe_check_errors.
#include "cluster_wait.cuh"
#include "device_util.cuh"
#include "launch.cuh"
#include "moe_internal.cuh"

namespace moe {

namespace {

__global__ void selftest_wait_kernel(int32_t *err, int polls)
{
    __shared__ uint64_t bar;
    __shared__ int abort;
    if (threadIdx.x == 0) {
        mbar_init(&bar, 1);
        abort = 0;
        fence_mbar_init();
    }
    __syncthreads();
    cluster_sync();
    pdl_wait();
    pdl_launch_dependents();
    // nothing arrives: the phase never completes and every poll fails
    if (blockIdx.x == 0 && threadIdx.x < 32) {
        wait_or_abort(&bar, 0, &abort, err, polls);
    } else {
        for (int left = polls / 4 + 64; left > 0 && !aborted(&abort); --left) {
            int turn = 64;
            poll(&bar, 0, turn);
        }
    }
    __syncthreads();
    cluster_sync();
}

}  // namespace

cudaError_t launch_selftest_wait(int32_t *err, int polls, cudaStream_t st)
{
    return launch_kernel(selftest_wait_kernel, dim3(2), dim3(64), 0, st, 2, err, polls);
}

}  // namespace moe
