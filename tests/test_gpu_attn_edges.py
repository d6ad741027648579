"""Attention over the paged cache at the edges of what a call may hold."""
import dataclasses

import pytest
import torch

import attn_cases as ac
import moe_expert_layer_sigmoid_gb300 as moe
from test_gpu_attn_paged import ok, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("end", [-2 ** 31, -2 ** 31 + 4, -1, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [4, 60])
def test_offsets_that_hold_anything(fmt, end, n):
    """Offsets whose difference does not fit 32 bits: the two sequences that share one are left out and
    recorded, the others are as ever."""
    b = ac.make([5, n, 3, 1, 40], [30, 70, 20, 50, 90], 8, 2, 64, 16, fmt, seed=3)
    b.q_off[2] = end
    out, lse, ws = run(b)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    ref, z, bo, bl = ac.reference(b)
    at = torch.tensor(list(range(5)) + list(range(8 + n, 49 + n)), device="cuda")
    assert ((out.double() - ref)[at].abs() <= bo[at]).all()
    assert ((lse.double() - z)[at].abs() <= bl[at]).all()
    assert (out[5:8 + n] == 7).all() and (lse[5:8 + n] == 7).all()


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30, 130, 3])
@pytest.mark.parametrize("G", [1, 4, 24])
def test_windows_with_tokens_before_the_start(fmt, window, G):
    """A window of any size, the largest standing for none, where some tokens sit before the start."""
    new = [10, 3, 1, 200, 40, 1]
    total = [5, 1, 0, 100, 17, 300]
    ok(ac.make(new, total, 2 * G, 2, 128, 16, fmt, window=window, seed=G))


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("new", [1, 3, 100, 250])
@pytest.mark.parametrize("page,left", [(64, 0), (64, 10), (16, 0), (16, 7)])
def test_the_longest_length(fmt, new, page, left):
    """Sequences that end within a tile of 2^31 keys, seen through a window; behind the last key of the page
    lies what must never matter."""
    far = 2 ** 31 - page          # keys of the longest page table
    total = far - left
    window, near = 300, 2048      # keys the window can reach, in whole pages
    b = ac.make([new], [near - left], 8, 2, 64, page, fmt, window=window, seed=new)
    # the same pages at the end of a page table of 2^31 keys: positions are 2^31 less a constant
    pages = torch.full((1, far // page), 0x7FFFFFF0, dtype=torch.int32, device="cuda")
    pages[0, -(near // page):] = b.pages[0, :near // page]
    ref = ac.reference(b)
    dims = b.dims(moe, max_pages=far // page)
    b.pages = pages
    b.kv_len.fill_(total)
    out, lse, ws = run(b, dims=dims)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    assert ((out.double() - ref[0]).abs() <= ref[2]).all()
    assert ((lse.double() - ref[1]).abs() <= ref[3]).all()


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("scale", [-0.3125, 0.0, -0.0, 1.0, -1.0, 2.0 ** -12, 2.0 ** -140])
@pytest.mark.parametrize("window", [0, 70])
@pytest.mark.parametrize("D", [64, 128])
def test_factors_of_the_scores(fmt, scale, window, D):
    """Any factor: a negative one turns the order of the scores, zero makes plain means; few rows and chunks,
    tokens before the start, a window, masks at every edge."""
    b = ac.make([1, 4, 90, 1, 20, 150], [300, 77, 200, 1, 9, 150], 8, 2, D, 16, fmt, window=window, seed=D)
    out, lse, ws = run(dataclasses.replace(b, scale=scale))
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    # the same scores from the other sign of the queries, so that the bounds' magnitudes stay positive
    ac.check(dataclasses.replace(b, scale=abs(scale), q=-b.q if scale < 0 else b.q), out, lse)


@pytest.mark.parametrize("fmt", ac.FORMATS)
def test_two_streams_at_once(fmt):
    """Calls at work at the same time on two streams, a workspace each, give what they give alone."""
    bs = [ac.make([1, 200, 3, 1], [3000, 900, 700, 50], 8, 2, 128, 16, fmt, seed=1),
          ac.make([150, 1, 1, 20], [400, 5000, 33, 20], 16, 2, 64, 32, fmt, seed=2)]
    alone = [run(b)[:2] for b in bs]
    wss = [moe.workspace(moe.moe_attn_workspace_bytes(b.dims(moe))) for b in bs]
    streams = [torch.cuda.Stream() for _ in bs]
    got = [[] for _ in bs]
    torch.cuda.synchronize()
    for _ in range(20):
        for i, b in enumerate(bs):
            with torch.cuda.stream(streams[i]):
                got[i].append(run(b, wss[i])[:2])
    torch.cuda.synchronize()
    for i, b in enumerate(bs):
        assert moe.moe_check_device_status(wss[i]) == moe.MOE_OK
        for out, lse in got[i]:
            assert torch.equal(out, alone[i][0]) and torch.equal(lse, alone[i][1])
        ac.check(b, *alone[i])


@pytest.mark.parametrize("fmt,tier", [("bf16", 10), ("bf16", 30), ("e4m3", 10), ("e4m3", 20), ("e4m3", 30),
                                      ("int4", 4), ("int4", 10)])
@pytest.mark.parametrize("D", [64, 128])
def test_queries_of_a_wide_range(fmt, tier, D):
    """One element of each query is 2^tier times the others and meets keys of 0, so the others make the scores:
    few rows of a coded cache hold them in f16, scaled to the largest, and sum shifted int4 codes."""
    b = ac.make([1, 2, 1, 40], [300, 77, 9, 90], 8, 2, D, 16, fmt, seed=D + tier)
    c = 6
    if fmt == "int4":
        b.k[..., c // 2] &= 0xF0
    else:
        b.k[..., c] = 0
    q = torch.randn(b.q.shape, generator=torch.Generator().manual_seed(tier)) * 2.0 ** -tier
    q[..., c] = 1.0
    b = dataclasses.replace(b, q=q.to(torch.bfloat16).cuda(), scale=2.0 ** (tier - 3))
    out, lse, ws = run(b)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    ref, z, bo, bl = ac.reference(b)
    # What the header states on top of the reference's bound: an element off by 2^-39 (int4: 2^-35) of the
    # largest, here 1, and int4 sums that round by |q| (|n| + 16) instead of |q n|.  `e` is the change of a score; a
    # weight moves by its own and the largest one's, numerator and denominator alike.
    k, v = (ac.values(x, None if s is None else s.nan_to_num(0.0), fmt).nan_to_num(0.0)
            for x, s in ((b.k, b.ks), (b.v, b.vs)))
    e = 0.0
    if fmt != "bf16":
        e = 2.0 ** (-39 if fmt == "e4m3" else -35) * k.abs().sum(-1).max().item() * b.scale
    if fmt == "int4":
        e += D * 2.0 ** -23 * 16 * b.ks.nan_to_num(0.0).max().item() * q.abs().sum(-1).max().item() * b.scale
    assert e < 0.1
    assert ((out.double() - ref).abs() <= bo + 4 * e * v.abs().max()).all()
    assert ((lse.double() - z).abs() <= bl + 2 * e).all()


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("G", [3, 5, 7, 24, 33, 100])
@pytest.mark.parametrize("D", [64, 128])
def test_same_bits_whatever_ran_before(fmt, G, D):
    """Groups that leave rows of a tile without a token: what other calls left in shared memory does not
    tell in the last bit."""
    b = ac.make([60, 1, 90], [700, 300, 1500], 2 * G, 2, D, 16, fmt, window=1000, seed=G)
    other = ac.make([300], [300], 16, 2, D, 16, fmt, seed=1)
    first, ws = None, moe.workspace(moe.moe_attn_workspace_bytes(b.dims(moe)))
    for factor in (1.0, 1e-3, 30.0, 1e4, -1e6, float("nan"), 0.0):
        run(dataclasses.replace(other, q=other.q * factor))
        out, lse, _ = run(b, ws)
        if first is None:
            first = out, lse
            ac.check(b, out, lse)
        assert torch.equal(out, first[0]) and torch.equal(lse, first[1]), factor
