"""Packed weights and codes that the binding makes itself are not in memory that the current stream still has to write."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from test_gpu_fp4_streams import busy

pytestmark = pytest.mark.gpu
ROWS, K = 2048, 4096


def blocks():
    g = torch.Generator().manual_seed(2)
    b = torch.randint(0, 256, (ROWS, K // 32, 18), generator=g, dtype=torch.uint8)
    b[..., 1] = 0x2C        # (a scale of 2^-4 or so)
    return b.view(ROWS, -1).cuda()


CALLS = {
    "moe_pack_w4": lambda s: moe.moe_pack_w4(torch.randn(ROWS, K, generator=torch.Generator().manual_seed(1)).cuda(), 64, stream=s),
    "moe_pack_w8": lambda s: moe.moe_pack_w8(torch.randn(ROWS, K, generator=torch.Generator().manual_seed(1)).cuda(), stream=s),
    "moe_quant_rows_fp8": lambda s: moe.moe_quant_rows_fp8(
        torch.randn(ROWS, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda(), stream=s),
    "moe_import_q4_blocks": lambda s: moe.moe_import_q4_blocks(blocks(), K, 64, stream=s),
}


@pytest.mark.parametrize("name", CALLS)
def test_outputs_made_for_another_stream(name, monkeypatch):
    made = []       # (inputs on the device before the stream is busy)
    real = getattr(moe, name)
    monkeypatch.setattr(moe, name, lambda *a, stream=None: made.append(a) or real(*a, stream=stream))
    want = CALLS[name](None)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    keep = busy()
    junk = [torch.empty_like(t) for t in want]
    for t in junk:
        t.view(torch.uint8).fill_(255)
    del junk, t
    got = real(*made[0], stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a.view(torch.uint8), b.view(torch.uint8))
    del keep
