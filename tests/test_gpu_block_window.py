"""A decoder block's steps whose sequences outgrow the window: pages go back on the way, and what they held never shows."""
import math
import os
import sys

import pytest
import torch

import attn_cases as ac

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt", ac.FORMATS)
def test_pages_that_the_window_gives_back(fmt, monkeypatch):
    import decode_step as ex
    moe, T = ex.moe, 40
    block = ex.Block(fmt, 3, T)
    k, v, ks, vs = block.pool
    attn = moe.moe_attn_paged
    seen = []

    def poison():
        """Every slot of a page that no sequence holds becomes what must never matter."""
        idle = torch.ones(ex.n_pages, dtype=torch.bool, device="cuda")
        idle[block.pages[block.pages >= 0].long()] = False
        for t in (k, v):
            t[idle] = math.nan if fmt == "bf16" else 0x7F
        for t in (ks, vs):
            if t is not None:
                t[idle] = math.nan

    def held_to_the_definition(q, q_off, kv_len, pages, dims, cache, scale, out, lse, ws):
        poison()
        n = q_off[-1].item()
        z = torch.full((dims.T, dims.H), 7.0, device="cuda")
        attn(q, q_off, kv_len, pages, dims, cache, scale, out, z, ws)
        ac.check(ac.Batch(q_off.diff().tolist(), kv_len.tolist(), dims.H, dims.H_kv, dims.D, dims.page, fmt, dims.window,
                          scale, q[:n], q_off, kv_len, pages, k, v, ks, vs), out[:n], z[:n])
        seen.append(block.first.tolist())

    monkeypatch.setattr(moe, "moe_attn_paged", held_to_the_definition)
    g = torch.Generator(device="cuda").manual_seed(3)
    # three chunks of a prompt, then tokens past the window's first pages; drafts dropped; an end and a new prompt
    steps = [[30, 5, 0], [30, 5, 0], [30, 5, 0], [20, 5, 0]] + [[1, 12, 1]] * 9 + [[4, 1, 1], [-3, 1, 1], [1, -(1 << 31), 1]] + \
            [[1, 30, 1], [1, 1, 30]] + [[1, 30, 3]] * 3
    length = [0, 0, 0]
    for new in steps:
        block.new.copy_(torch.tensor(new, dtype=torch.int32))
        block.residual.copy_(torch.randn((T, ex.d), generator=g, device="cuda").to(torch.bfloat16))
        block.step()
        assert block.status() == [moe.MOE_OK] * 3
        before, length = length, [max(0, n + m) for n, m in zip(length, new)]
        assert block.kv_len.tolist() == length
        n = sum(m for m in new if m > 0)
        assert torch.isfinite(block.residual[:n].float()).all()
        # a sequence holds the pages from the one that its next token sees first, and every page is held or free
        for b in range(3):
            if new[b] >= 0:
                assert block.first[b].item() == max(0, before[b] - ex.window + 1) // ex.page
            held = (block.pages[b] >= 0).nonzero().view(-1).tolist()
            assert held == list(range(block.first[b].item(), -(-length[b] // ex.page)))
        ids = torch.cat((block.pages[block.pages >= 0], block.free[:block.n_free.item()])).tolist()
        assert sorted(ids) == list(range(ex.n_pages))
    assert max(f[0] for f in seen) >= 1 and max(f[1] for f in seen) >= 1


def test_captured_steps_past_the_window():
    """The same lengths as a replayed graph: outputs and states equal to plain steps'."""
    import decode_step as ex
    T = 40
    eager, graphed = ex.Block("e4m3", 3, T), ex.Block("e4m3", 3, T)
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    graphed.step()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream), torch.cuda.graph(graph, stream=stream):
        graphed.step()
    g = torch.Generator(device="cuda").manual_seed(4)
    for new in [[38, 1, 1]] * 3 + [[1, 36, 1]] * 4 + [[-1, 1, 30]] + [[1, 1, 1]] * 20:
        x = torch.randn((T, ex.d), generator=g, device="cuda").to(torch.bfloat16)
        n = sum(m for m in new if m > 0)
        for block in (eager, graphed):
            block.new.copy_(torch.tensor(new, dtype=torch.int32))
            block.residual.copy_(x)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.residual[:n], graphed.residual[:n])
        for a, b in zip(eager.held.tensors, graphed.held.tensors):
            assert torch.equal(a, b)
    assert eager.status() == graphed.status() == [ex.moe.MOE_OK] * 3
    assert eager.first.tolist()[0] >= 1 and eager.first.tolist()[1] >= 1
