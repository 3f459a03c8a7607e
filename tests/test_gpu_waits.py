"""The bounded device-side waits of kernels whose CTAs wait for one another, made to run out."""
import time

import pytest
import torch

import sparse_expert_ffn_route_gb300 as moe

pytestmark = pytest.mark.gpu


def test_a_wait_that_gives_up_ends_the_whole_cluster():
    """One warp of a pair of CTAs gives up after a few polls; three others, which go on sixteen times
    as long by themselves, end with it, and the workspace is usable again."""
    ws = moe.alloc_mxfp4_matmul_workspace()
    moe.moe_selftest_wait_timeout(ws, polls=64)
    with pytest.raises(moe.MoeError) as e:
        moe.moe_check_errors(ws)
    assert e.value.code == moe.MOE_ERR_TIMEOUT
    began = time.perf_counter()
    moe.moe_selftest_wait_timeout(ws, polls=1 << 14)          # 62 ms
    torch.cuda.synchronize()
    assert time.perf_counter() - began < 0.5
    with pytest.raises(moe.MoeError):
        moe.moe_check_errors(ws)
    moe.moe_check_errors(ws)
