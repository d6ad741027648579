"""The norms between blocks against their formulas in 64 bits, element by element."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu
EPS = 1e-6


def formula(y, res, gate, w_post, w_pre, kind, sigmoid, scale):
    """r', x and the size of the terms that meet in r', in 64 bits."""
    d = lambda t: None if t is None else t.double().cpu()  # noqa: E731
    y, res, gate, w_post, w_pre = map(d, (y, res, gate, w_post, w_pre))
    r, size = res, res.abs()
    if y is not None:
        u = y
        if w_post is not None:
            u = u / (u.square().mean(-1, keepdim=True) + EPS).sqrt() * w_post
        if gate is not None:
            g = gate[:, None] if kind == moe.MOE_GATE_TOKEN else gate
            u = u * (1 / (1 + torch.exp(-g)) if sigmoid else g)
        r = res + scale * u
        size = res.abs() + (scale * u).abs()
    x = None if w_pre is None else r / (r.square().mean(-1, keepdim=True) + EPS).sqrt() * w_pre
    return r, x, size


def inputs(T, d, kind, post, pre, res32, seed=0, y=True):
    g = torch.Generator().manual_seed(seed)
    n = lambda *s: torch.randn(s, generator=g)  # noqa: E731
    gate = {0: None, 1: n(T), 2: n(d), 3: n(T, d).to(torch.bfloat16)}[kind]
    got = (n(T, d).to(torch.bfloat16) if y else None, (3 * n(T, d)).to(torch.float32 if res32 else torch.bfloat16), gate,
           1 + 0.2 * n(d) if post else None, 1 + 0.2 * n(d) if pre else None)
    return [None if t is None else t.cuda() for t in got]


def check(y, res, gate, w_post, w_pre, dims, r_out, x):
    kind, d = dims.gate, dims.d
    r, xw, size = formula(y, res, gate, w_post, w_pre, kind, dims.flags & moe.MOE_NORM_SIGMOID, dims.scale)
    # fp32 steps: a sum of d squares in any tree that the kernel takes (at most 32 + 12 additions deep per
    # term, 2^-24 each, half of it in the root), the root (2^-22), the gate's exponential (2^-21 for |g| < 8) and some products
    f32 = 2.0 ** -18
    if y is not None:
        half = 2.0 ** -24 if dims.flags & moe.MOE_NORM_RESIDUAL_F32 else 2.0 ** -8
        fine = (r_out.double().cpu() - r).abs() <= half * r.abs() + f32 * size + 1e-37
        assert fine.all()
    if xw is not None:
        # (what the terms lost before they cancel counts against the row's root mean square)
        rms = (r.square().mean(-1, keepdim=True) + EPS).sqrt()
        room = f32 * (xw.abs() + (size / rms) * w_pre.double().cpu().abs())
        fine = (x.double().cpu() - xw).abs() <= 2.0 ** -8 * xw.abs() + 2 * room + 1e-37
        assert fine.all()


def run(args, dims, in_place=False):
    y, res, gate, w_post, w_pre = args
    keep = [None if t is None else t.clone() for t in args]
    r_out = res if in_place else torch.full_like(res, 7.0)
    x = None if w_pre is None else y if in_place and y is not None else torch.full(res.shape, 7.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_block_norm(y, res, gate, w_post, w_pre, dims, r_out, x)
    check(*keep, dims, r_out, x)
    return r_out, x


@pytest.mark.parametrize("kind", [0, 1, 2, 3])
@pytest.mark.parametrize("post,pre", [(True, True), (False, True), (True, False), (False, False)])
@pytest.mark.parametrize("T,d", [(1, 8), (3, 264), (9, 520), (2, 1024), (5, 1032), (1, 4096), (33, 5000)])
def test_parts(T, d, kind, post, pre):
    for res32 in (False, True):
        dims = moe.NormDims(T=T, d=d, gate=kind, flags=(moe.MOE_NORM_RESIDUAL_F32 if res32 else 0) | (moe.MOE_NORM_SIGMOID if T % 2 else 0),
                            eps=EPS, scale=0.7)
        run(inputs(T, d, kind, post, pre, res32, seed=d + kind), dims)


@pytest.mark.parametrize("d", [8, 248, 256, 504, 512, 768, 1016, 1024, 1032, 2048, 2056, 4088, 4104, 8192, 8200, 16384, 16392, 24584, 32768])
@pytest.mark.parametrize("res32", [False, True])
def test_widths(d, res32):
    dims = moe.NormDims(T=7, d=d, gate=3, flags=moe.MOE_NORM_RESIDUAL_F32 if res32 else 0, eps=EPS, scale=-1.25)
    run(inputs(7, d, 3, True, True, res32, seed=d), dims)
    run(inputs(7, d, 3, True, True, res32, seed=d + 1), dims, in_place=True)


@pytest.mark.parametrize("T,d", [(20000, 64), (3001, 2048), (70000, 8)])
def test_many_rows(T, d):
    dims = moe.NormDims(T=T, d=d, gate=1, flags=0, eps=EPS, scale=1.0)
    run(inputs(T, d, 1, True, True, False), dims)


@pytest.mark.parametrize("T,d", [(1, 4096), (5, 256), (3, 9000)])
def test_the_first_norm(T, d):
    _, res, _, _, w_pre = inputs(T, d, 0, False, True, False, y=False)
    dims = moe.NormDims(T=T, d=d, gate=0, flags=0, eps=EPS, scale=1.0)
    x = torch.empty(T, d, dtype=torch.bfloat16, device="cuda")
    was = res.clone()
    moe.moe_block_norm(None, res, None, None, w_pre, dims, None, x)
    check(None, was, None, None, w_pre, dims, None, x)
    assert torch.equal(res, was)
    moe.moe_block_norm(None, res, None, None, w_pre, dims, res, x)     # (an output that is not written)
    assert torch.equal(res, was)


def test_rows_of_zeros_and_large_gates():
    dims = moe.NormDims(T=3, d=512, gate=1, flags=moe.MOE_NORM_SIGMOID, eps=EPS, scale=1.0)
    y, res, gate, w_post, w_pre = inputs(3, 512, 1, True, True, False)
    y[0], res[0] = 0, 0
    gate.copy_(torch.tensor([0.0, -200.0, 200.0]))
    r, x = run((y, res, gate, w_post, w_pre), dims)
    assert (r[0] == 0).all() and (x[0] == 0).all() and torch.equal(r[1], res[1])


def test_same_bits_every_time_and_beside_other_rows():
    args = inputs(600, 4096, 3, True, True, False)
    dims = moe.NormDims(T=600, d=4096, gate=3, flags=0, eps=EPS, scale=1.0)
    r, x = run(args, dims)
    r2, x2 = run(args, dims)
    assert torch.equal(r, r2) and torch.equal(x, x2)
    one = [args[0][17:18], args[1][17:18], args[2][17:18], args[3], args[4]]
    r1, x1 = run(one, moe.NormDims(T=1, d=4096, gate=3, flags=0, eps=EPS, scale=1.0))
    assert torch.equal(r1[0], r[17]) and torch.equal(x1[0], x[17])


def test_no_rows():
    dims = moe.NormDims(T=0, d=256, gate=1, flags=0, eps=EPS, scale=1.0)
    e = torch.empty(0, 256, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(256, device="cuda")
    moe.moe_block_norm(e, e, torch.empty(0, device="cuda"), w, w, dims, e, e)


def test_captured_on_another_stream():
    args = inputs(50, 4096, 2, True, True, False)
    dims = moe.NormDims(T=50, d=4096, gate=2, flags=0, eps=EPS, scale=1.0)
    r, x = run(args, dims)
    r2, x2 = torch.zeros_like(r), torch.zeros_like(x)
    s, g = torch.cuda.Stream(), torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.stream(s), torch.cuda.graph(g, stream=s):
        moe.moe_block_norm(*args, dims, r2, x2)
    for _ in range(2):
        r2.zero_()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(r, r2) and torch.equal(x, x2)


def test_the_binding_refuses():
    y, res, gate, w_post, w_pre = inputs(4, 256, 0, True, True, False)
    dims = moe.NormDims(T=4, d=256, gate=0, flags=0, eps=EPS, scale=1.0)
    out, x = torch.empty_like(res), torch.empty_like(y)
    for args in ((y[:3], res, None, w_post, w_pre), (y, res.float(), None, w_post, w_pre), (y.half(), res, None, w_post, w_pre),
                 (y, res, None, w_post.cpu(), w_pre), (y, res, None, w_post[:128], w_pre), (y.t(), res, None, w_post, w_pre),
                 (y, res, None, w_post, w_pre.to(torch.bfloat16))):
        with pytest.raises(ValueError):
            moe.moe_block_norm(*args, dims, out, x)
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm(y, res, None, w_post, w_pre, dims, out, None)
    with pytest.raises(moe.MoeError):
        moe.moe_block_norm(y, res, res, w_post, w_pre, dims, out, x)
