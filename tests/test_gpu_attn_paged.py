"""Attention of new tokens over the paged cache against its definition in 64 bits, element by
element within the bound that the stated numerics give (tests/attn_cases.py)."""
import math

import pytest
import torch

import attn_cases as ac
import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


def run(b, ws=None, dims=None, stream=None, lse=True):
    dims = dims or b.dims(moe)
    ws = moe.workspace(moe.moe_attn_workspace_bytes(dims)) if ws is None else ws
    out = torch.full((dims.T, b.H, b.D), 7.0, dtype=torch.bfloat16, device="cuda")
    z = torch.full((dims.T, b.H), 7.0, device="cuda") if lse else None
    moe.moe_attn_paged(b.q, b.q_off, b.kv_len, b.pages, dims, b.cache(moe), b.scale, out, z, ws,
                       stream=stream)
    return out, z, ws


def ok(b, **kw):
    out, lse, ws = run(b, **kw)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    ac.check(b, out, lse)
    return out, lse


SHAPES = [  # H, H_kv, D, page, layout
    (1, 1, 64, 16, "heads"), (8, 2, 128, 16, "tokens"), (7, 1, 128, 64, "heads"),
    (28, 4, 64, 32, "strided"), (16, 1, 128, 128, "heads"), (40, 8, 128, 256, "tokens"),
    (33, 1, 64, 64, "heads"), (128, 1, 128, 16, "heads"),
]


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("H,H_kv,D,page,layout", SHAPES)
def test_single_tokens(fmt, H, H_kv, D, page, layout):
    """One token per sequence at lengths around pages and tiles, idle slots among them."""
    total = [1, 2, 15, 16, 17, 0, 63, 64, 65, 127, 128, 129, 300, 0, 1025]
    new = [0 if t == 0 else 1 for t in total]
    ok(ac.make(new, total, H, H_kv, D, page, fmt, layout=layout, seed=H))


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("H,H_kv,D,page,layout", SHAPES)
def test_chunks(fmt, H, H_kv, D, page, layout):
    """Chunks of 1 to a few hundred tokens, after nothing or after earlier tokens."""
    new = [1, 5, 0, 33, 130, 2, 200]
    total = [1, 5, 0, 97, 130, 513, 333]
    if H >= 40:
        new, total = new[:4] + [65], total[:4] + [200]
    ok(ac.make(new, total, H, H_kv, D, page, fmt, layout=layout, seed=H + 1))


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("window", [1, 2, 16, 63, 64, 100, 128, 1000])
@pytest.mark.parametrize("D", [64, 128])
def test_window(fmt, window, D):
    """A sliding window: keys before it are not read, nor their pages."""
    new = [1, 7, 1, 90, 1, 3]
    total = [600, 200, 64, 300, 65, 3]
    ok(ac.make(new, total, 6, 2, D, 16, fmt, window=window, seed=window))


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("G", [1, 4, 24])
def test_tokens_that_see_nothing(fmt, G):
    """kv_len below the number of new tokens: the first of them sit before the start and see no
    key; out is 0 and lse -inf there, the others are as ever."""
    new = [3, 40, 1, 200, 6]
    total = [1, 17, 0, 5, 6]
    b = ac.make(new, total, 2 * G, 2, 128, 16, fmt, seed=G)
    out, lse = ok(b)
    assert (out[:2] == 0).all() and torch.isinf(lse[:2]).all()
    assert (out[43] == 0).all() and lse[43].eq(-math.inf).all()


@pytest.mark.parametrize("fmt", ac.FORMATS)
def test_peaked_and_flat_scores(fmt):
    """Scores hundreds apart (one key takes all the weight, its place anywhere), and all alike."""
    for spread, seed in ((60.0, 1), (0.0, 2)):
        b = ac.make([1, 2, 40, 1], [700, 130, 390, 64], 8, 2, 128, 32, fmt, spread=spread, seed=seed)
        ok(b)


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("new,total", [([1], [20011]), ([4], [9001]), ([70], [6000]), ([1, 300], [5000, 4001])])
def test_long_contexts(fmt, new, total):
    """Caches long enough to be split over many CTAs and joined."""
    ok(ac.make(new, total, 16, 2, 128, 64, fmt, seed=total[0]))


def test_zero_scales_and_zero_queries():
    """Rows of zeros in the cache (scale 0) and queries of zeros: plain means, no NaN."""
    b = ac.make([1, 30], [100, 64], 4, 1, 64, 16, "int4", poison=False)
    b.ks[::2] = 0
    b.vs[1::2] = 0
    b.q[0] = 0
    ok(b)


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pool_past_32_bits(fmt):
    """Pages whose byte offsets pass 2^32."""
    first = (1 << 33) // (8 * 256 * 128 * 2) if fmt == "bf16" else (1 << 32) // (8 * 256 * 128)
    b = ac.make([1, 50], [700, 300], 8, 8, 128, 256, fmt, first_page=first, seed=5)
    assert b.k.stride(0) * b.k.element_size() * b.pages[0, 0].item() >= 1 << 32
    ok(b)


@pytest.mark.parametrize("new", [[1] * 700, [0] * 300 + [1, 9, 0, 40] + [0] * 1200])
def test_many_sequences(new):
    total = [n and n + (37 * i) % 90 for i, n in enumerate(new)]
    ok(ac.make(new, total, 4, 2, 64, 16, "bf16", seed=9))


def test_max_new_is_only_a_hint():
    """The same values to the stated numerics whatever max_new says."""
    b = ac.make([1, 2, 60, 1], [50, 400, 60, 900], 12, 4, 128, 16, "bf16", seed=3)
    for hint in (0, 1, 60, 5000):
        ok(b, dims=b.dims(moe, max_new=hint))


def test_same_bits_again_and_workspace_reuse():
    """Same inputs, same bits; one workspace serves calls of different shapes in turn."""
    big = ac.make([1, 1, 20, 130], [4000, 900, 700, 1300], 16, 4, 128, 16, "e4m3", seed=1)
    small = ac.make([1], [37], 8, 2, 64, 32, "bf16", seed=2)
    ws = moe.workspace(max(moe.moe_attn_workspace_bytes(x.dims(moe)) for x in (big, small)))
    first = run(big, ws)[:2], run(small, ws)[:2]
    for _ in range(3):
        again = run(big, ws)[:2], run(small, ws)[:2]
        for (o1, z1), (o2, z2) in zip(first, again):
            assert torch.equal(o1, o2) and torch.equal(z1, z2)
    ac.check(big, *first[0])
    ac.check(small, *first[1])


def test_without_lse_and_on_another_stream():
    b = ac.make([1, 80], [300, 200], 8, 2, 128, 16, "bf16", seed=4)
    st = torch.cuda.Stream()
    torch.cuda.synchronize()
    out, _, ws = run(b, stream=st, lse=False)
    st.synchronize()
    want, lse, _ = run(b)
    assert torch.equal(out, want)
    ac.check(b, out, lse)


def test_graph_replay_follows_the_lengths():
    """A captured call reads lengths, offsets and pages when it runs."""
    b = ac.make([1, 1, 1], [100, 900, 33], 8, 2, 128, 16, "int4", seed=6)
    out, lse, ws = run(b)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_attn_paged(b.q, b.q_off, b.kv_len, b.pages, b.dims(moe), b.cache(moe), b.scale, out,
                           lse, ws)
    b.total = [64, 17, 33]
    b.kv_len.copy_(torch.tensor(b.total, dtype=torch.int32))
    b.q.mul_(0.5)
    g.replay()
    torch.cuda.synchronize()
    ac.check(b, out, lse)


def test_device_checks():
    """Bad lengths, offsets and page ids are recorded; the sound sequences are as ever."""
    b = ac.make([1, 30, 1, 4], [100, 90, 50, 44], 8, 2, 64, 16, "bf16", poison=False, seed=7)
    keep = b.kv_len.clone()
    b.kv_len[0] = b.pages.shape[1] * 16 + 1
    out, lse, ws = run(b)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    ref = ac.reference(b)
    assert ((out.double() - ref[0])[1:].abs() <= ref[2][1:]).all()
    b.kv_len[0] = -1
    out, lse, ws = run(b)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert ((out.double() - ref[0])[1:].abs() <= ref[2][1:]).all()
    b.kv_len.copy_(keep)
    off = b.q_off.clone()
    b.q_off[2] = 37                      # sequence 1 ends past the batch, 2 is descending
    out, lse, ws = run(b)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert ((out.double() - ref[0])[32:].abs() <= ref[2][32:]).all()
    b.q_off.copy_(off)
    page = b.pages.clone()
    b.pages[2, 1] = -5
    b.pages[2, 2] = b.k.shape[0]
    out, lse, ws = run(b)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    b.pages.copy_(page)
    ok(b)


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("stage", [1, 2])
@pytest.mark.parametrize("new,total", [([1], [200000]), ([100, 70], [900, 300]), ([1, 200, 1], [500, 700, 90])])
def test_a_wait_that_runs_out(fmt, stage, new, total):
    """A stage whose copies never come: every role gives up in order, the status says so, and the
    workspace serves the next call as a fresh one does."""
    b = ac.make(new, total, 8, 2, 128, 64, fmt, seed=5)
    dims = b.dims(moe)
    ws = moe.workspace(moe.moe_attn_workspace_bytes(dims))
    moe.moe_debug_set_waits(ws, 5_000_000, stage)
    run(b, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    moe.moe_debug_set_waits(ws, 0, 0)
    out, lse, _ = run(b, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    fresh, z, _ = run(b)
    assert torch.equal(out, fresh) and torch.equal(lse, z)
    ac.check(b, out, lse)


def test_binding_refuses():
    b = ac.make([1, 3], [20, 30], 4, 2, 64, 16, "e4m3", poison=False)
    d, c, ws = b.dims(moe), b.cache(moe), moe.workspace(moe.moe_attn_workspace_bytes(b.dims(moe)))
    out = torch.empty((4, 4, 64), dtype=torch.bfloat16, device="cuda")

    def call(q=b.q, off=b.q_off, lens=b.kv_len, pages=b.pages, dims=d, o=out, lse=None):
        moe.moe_attn_paged(q, off, lens, pages, dims, c, 0.1, o, lse, ws)

    call()
    for kw in (dict(q=b.q[:3]), dict(q=b.q.float()), dict(q=b.q.transpose(0, 1)), dict(off=b.q_off[:2]),
               dict(lens=b.kv_len.long()), dict(pages=b.pages[:1]), dict(o=out[:3]),
               dict(lse=torch.empty(3, device="cuda")), dict(dims=d.replace(page=32)),
               dict(o=out.cpu())):
        with pytest.raises(ValueError):
            call(**kw)
    with pytest.raises(moe.MoeError):
        call(dims=d.replace(window=-1))
