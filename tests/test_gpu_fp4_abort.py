"""Projections by pairs of CTAs whose leader misses a stage: the call ends with the status, whether every copy was issued before
the first wait or stages had come round, and the workspace serves the next call."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


# one tile to a pair with at most as many stages of 256 as there are places (5), one more, many; several tiles to a pair
@pytest.mark.parametrize("T,N,K,stages", [(1024, 2560, 256, [1]), (1024, 2560, 1024, [1, 4]), (1024, 2560, 1280, [5]), (1024, 2560, 1536, [2, 6]),
                                          (1024, 2560, 8192, [3, 32]), (2000, 6144, 512, [1, 4, 6])])
def test_a_stage_that_never_comes(T, N, K, stages):
    g = torch.Generator().manual_seed(K)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    w = moe.fp4(*moe.moe_pack_fp4(torch.randn(N, K, generator=g).cuda()))
    ws = moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K))
    out, want = (torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_linear_fp4(x, w, want, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    for stage in stages:
        moe.moe_debug_set_waits(ws, 1_000_000, stage)     # 1 ms: every other wait of these launches takes microseconds
        moe.moe_linear_fp4(x, w, out, ws)
        assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
        # tiles of other pairs are as always: the first pair's first tile is tokens 0 to 255 of channels 0 to 255
        assert torch.equal(out[256:512, :256], want[256:512, :256])
        moe.moe_debug_set_waits(ws, 0, 0)
        out.zero_()
        moe.moe_linear_fp4(x, w, out, ws)
        assert moe.moe_check_device_status(ws) == moe.MOE_OK and torch.equal(out, want)
