"""The fused rotary write as a decode step calls it: queries in place in the projection's buffer, captured and replayed with
other positions and slots, two streams at work at once, positions of any order and the same one many times."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from attn_cases import FORMATS
from test_gpu_rope import _write_setup, table_of

pytestmark = pytest.mark.gpu


def pool_of(pool, sc):
    return [t for t in (*pool, *sc) if t is not None]


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("T,H,H_kv,D,rot", [(1, 32, 8, 128, 128), (37, 7, 1, 64, 48), (3000, 12, 4, 128, 64), (20000, 3, 3, 64, 64)])
def test_in_place(T, H, H_kv, D, rot, norm, fmt):
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(T, H, H_kv, D, 32, fmt, "heads", seed=T)
    pos[::9], slots[::7] = -1, -1
    pos[1::3] = 1999                    # (one position of many tokens)
    pos, slots, table, ws = pos.cuda(), slots.cuda(), table_of(2000, rot), moe.workspace(256)
    g = torch.Generator().manual_seed(5)
    w = [torch.randn(D, generator=g).cuda() if norm else None for _ in range(2)]
    r = moe.rope(table, moe.MOE_ROPE_PAIRS if T % 2 else 0, *w, 1e-6)
    out = q.clone()                     # (tokens that are left out keep what is there)
    moe.moe_rope_kv_write(q, k, v, pos, slots, r, dims, cache, out, ws)
    want = [t.clone() for t in pool_of(pool, sc)]
    for t in pool_of(pool, sc):
        t.fill_(3)
    moe.moe_rope_kv_write(q, k, v, pos, slots, r, dims, cache, out.clone(), ws)   # (what the pools are where nothing is written)
    base = [t.clone() for t in pool_of(pool, sc)]
    for t in pool_of(pool, sc):
        t.fill_(3)
    k_was, v_was = k.clone(), v.clone()
    moe.moe_rope_kv_write(q, k, v, pos, slots, r, dims, cache, q, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    assert torch.equal(q, out) and torch.equal(k, k_was) and torch.equal(v, v_was)
    assert all(torch.equal(a, b) for a, b in zip(pool_of(pool, sc), base))
    live = (pos >= 0) & (slots >= 0)
    p, at = slots[live].long() // 32, slots[live].long() % 32
    assert all(torch.equal(a[p, :, at], b[p, :, at]) for a, b in zip(base, want))


@pytest.mark.parametrize("fmt", FORMATS)
def test_captured_and_on_two_streams(fmt):
    T, H, H_kv, D = 300, 8, 2, 128
    sets = [_write_setup(T, H, H_kv, D, 16, fmt, "heads", seed=s) for s in (1, 2)]
    table = table_of(2000, D)
    r = moe.rope(table, 0, torch.ones(D, device="cuda"), torch.ones(D, device="cuda"), 1e-6)
    runs = []
    for q, k, v, slots, pos, pool, sc, dims, cache in sets:
        at = [t.cuda() for t in (pos, slots)]
        out, ws, s, graph = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda"), moe.workspace(256), torch.cuda.Stream(), torch.cuda.CUDAGraph()
        torch.cuda.synchronize()
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            moe.moe_rope_kv_write(q, k, v, *at, r, dims, cache, out, ws)
        runs.append((q, k, v, pos, slots, pool, sc, dims, cache, at, out, ws, s, graph))
    for turn in range(3):
        wants = []
        for q, k, v, pos, slots, pool, sc, dims, cache, at, out, ws, s, graph in runs:
            at[0].copy_((pos * (turn + 1) + 7 * turn) % 2000)
            at[1].copy_(slots.roll(turn))
            want = torch.empty_like(out)
            moe.moe_rope_kv_write(q, k, v, *at, r, dims, cache, want, ws)
            wants.append([want] + [t.clone() for t in pool_of(pool, sc)])
            out.zero_()
            for t in pool_of(pool, sc):
                t.fill_(3)
        torch.cuda.synchronize()
        for _ in range(5):
            for run in runs:
                with torch.cuda.stream(run[12]):
                    run[13].replay()
        torch.cuda.synchronize()
        for (q, k, v, pos, slots, pool, sc, dims, cache, at, out, ws, s, graph), want in zip(runs, wants):
            assert torch.equal(out, want[0]) and moe.moe_check_device_status(ws) == moe.MOE_OK
            p, where = at[1].long() // 16, at[1].long() % 16
            for a, b in zip(pool_of(pool, sc), want[1:]):
                assert torch.equal(a[p, :, where], b[p, :, where])
