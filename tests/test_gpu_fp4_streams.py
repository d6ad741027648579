"""Outputs that the binding makes itself belong to the stream of the call: nothing that the current stream still has to do gets
between them and the kernel."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


def busy():
    """Some milliseconds of work for the current stream."""
    t = torch.empty(1 << 30, dtype=torch.uint8, device="cuda")
    for i in range(30):
        t.fill_(i)
    return t


@pytest.mark.parametrize("rows,K", [(1, 64), (300, 1024), (5, 20480)])
@pytest.mark.parametrize("half", [True, False])
def test_outputs_made_for_another_stream(rows, K, half):
    g = torch.Generator().manual_seed(rows)
    x = torch.randn(rows, K, generator=g).to(torch.bfloat16 if half else torch.float32).cuda()
    f = moe.moe_quant_rows_fp4 if half else moe.moe_pack_fp4
    want = f(x)
    back = moe.moe_unpack_fp4(*want)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = busy()
    got = f(x, stream=s)
    out = moe.moe_unpack_fp4(*got, stream=s)
    torch.cuda.synchronize()
    for a, b in zip((*got, out), (*want, back)):
        assert torch.equal(a, b)
    del keep


def test_memory_that_the_current_stream_still_uses():
    """A block that was freed with work on it pending is not handed to the other stream."""
    x = torch.randn(4096, 4096, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    want = moe.moe_quant_rows_fp4(x)
    s = torch.cuda.Stream()
    torch.cuda.synchronize()
    keep = busy()
    junk = torch.empty_like(want[0])      # the size of the codes
    junk.fill_(255)                       # behind all of that
    del junk
    got = moe.moe_quant_rows_fp4(x, stream=s)
    torch.cuda.synchronize()
    for a, b in zip(got, want):
        assert torch.equal(a, b)
    del keep
