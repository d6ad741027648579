"""Projections whose scale tiles hold NaN for rows past the last, in the weights and in what a workspace was left with: nothing of it
reaches an output, and nothing is written past the outputs or the workspace."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from test_gpu_fp4 import check, rows_of, written

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T,N,K", [
    (1, 8, 64), (1, 6152, 4096), (2, 136, 448), (2, 8200, 4160), (3, 8, 64), (5, 264, 8256), (17, 1000, 320), (33, 72, 1088), (64, 136, 16448),
    (65, 8, 128), (100, 200, 4160), (130, 1032, 832), (300, 264, 8192), (500, 10248, 192), (1100, 2568, 1344), (129, 20008, 64),
])
def test_rows_past_the_last_hold_nan(T, N, K):
    g = torch.Generator().manual_seed(T + N + K)
    x = rows_of(T, K, "outliers", seed=T).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g) / K ** 0.5
    q, b, s = moe.moe_pack_fp4(w.cuda())
    b[~written(N, K).cuda()] = 0x7F
    need = moe.moe_linear_fp4_workspace_bytes(T, N, K)
    space = torch.full((need + 512,), 0xFF, dtype=torch.uint8, device="cuda")
    space[:256] = 0                         # (the header; behind it what earlier calls left)
    buf = torch.full((T + 300, N), 7.0, dtype=torch.bfloat16, device="cuda")
    for _ in range(2):
        moe.moe_linear_fp4(x.cuda(), moe.fp4(q, b, s), buf[:T], space[:need])
    assert moe.moe_check_device_status(space[:need]) == moe.MOE_OK
    check(buf[:T], x, w)
    assert (buf[T:] == 7).all() and (space[need:] == 0xFF).all()
    # the weights themselves are only read
    again = moe.moe_pack_fp4(w.cuda())
    assert torch.equal(q, again[0]) and torch.equal(s, again[2]) and (b[~written(N, K).cuda()] == 0x7F).all()
