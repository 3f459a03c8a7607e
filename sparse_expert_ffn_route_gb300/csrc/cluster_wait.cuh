// cluster_wait.cuh -- bounded waits of kernels whose CTAs depend on one another (a cluster's, a
// pair's), and how one that gives up ends all of them.
//
// A warp waits on an mbarrier for kClusterWaitLimit polls at most: one second on GB300, where a poll of
// a barrier that nothing arrives at takes 3.8 us; the longest wait of these kernels, a tile's whole
// reduction, is under a millisecond.  One that gives up records kErrTimeout in the workspace's error
// word, sets `abort` in the shared memory of every CTA of its cluster and leaves its loops; every
// warp looks at `abort` between tiles.  After a lost arrival all warps that depend on it are waiting
// within microseconds, so their limits run out together and the kernel ends after about one.  (The CTAs of a
// cluster end together, behind a cluster barrier, so the others' memory is there to be written.)
//
// The poll loop does not look at `abort`: its few instructions lie on the path from one stage to the
// next, and a look between polls cost a prompt's product 60 -> 72 us and its expert block 953 -> 1146.
//
// What a kernel has in flight when it stops like that (copies and other CTAs' stores into its shared
// memory, MMAs on its tensor memory) completes by itself in microseconds, but nothing says when: settle()
// has every CTA wait 15 ms before it goes to the barrier behind which they end.
#pragma once

#include "device_util.cuh"
#include "moe_internal.cuh"

namespace moe {

constexpr int kClusterWaitLimit = 1 << 18;
constexpr int kSettleLimit = 1 << 12;   // polls

__device__ __forceinline__ uint32_t map_rank(uint32_t saddr, int rank)
{
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync()
{
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}

// mbar_try_wait on a barrier that other CTAs of the cluster arrive at (their writes become visible)
__device__ __forceinline__ bool mbar_try_wait_cluster(uint64_t *bar, uint32_t parity)
{
    uint32_t ok;
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(ok)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return ok != 0;
}

// by a whole warp; false once any of its lanes gave up
template <bool CLUSTER = false>
__device__ __forceinline__ bool wait_or_abort(uint64_t *bar, uint32_t parity, int *abort, int32_t *err, int limit = kClusterWaitLimit)
{
    bool ok = false;
    for (int n = 0; n < limit; ++n) {
        ok = CLUSTER ? mbar_try_wait_cluster(bar, parity) : mbar_try_wait(bar, parity);
        if (ok) break;
    }
    ok = __all_sync(0xffffffffu, ok);
    if (!ok) {
        uint32_t lane, ctas;
        asm("mov.u32 %0, %%laneid;" : "=r"(lane));
        asm("mov.u32 %0, %%cluster_nctarank;" : "=r"(ctas));
        if (lane == 0) atomicOr(err, kErrTimeout);
        if (lane < ctas)
            asm volatile("st.relaxed.cluster.shared::cluster.u32 [%0], 1;" ::"r"(map_rank(smem_u32(abort), (int)lane)) : "memory");
        __syncwarp();
    }
    return ok;
}

// (a vote, so that loops on it are uniform across the warp for the compiler too)
__device__ __forceinline__ bool aborted(const int *abort)
{
    return __any_sync(0xffffffffu, *(volatile const int *)abort != 0);
}

// waits for a phase without recording anything; `polls` is what is left of the limit
__device__ __forceinline__ void poll(uint64_t *bar, uint32_t parity, int &polls)
{
    while (polls > 0 && !mbar_try_wait(bar, parity)) --polls;
}

// By one warp of each CTA at its end: waits for the first phase of `fin`, the commit of all MMAs, and
// after a stop for the rest of the limit too (no second phase follows).
__device__ __forceinline__ void settle(uint64_t *fin, const int *abort)
{
    int polls = kSettleLimit;
    poll(fin, 0, polls);
    if (aborted(abort)) poll(fin, 1, polls);
    __syncwarp();
}

}  // namespace moe
