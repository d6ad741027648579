"""4-bit floats: codes, block scales and row scales equal to the recipe bit for bit, and projections against
the sums of what the codes stand for in 64 bits."""
import math

import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu
SIZES = torch.tensor([0, 0.5, 1, 1.5, 2, 3, 4, 6], dtype=torch.float64)


def e4m3_values():
    v = torch.arange(127)
    e, f = v >> 3, (v & 7).double()
    return torch.where(e == 0, f * 2.0 ** -9, (8 + f) * torch.exp2(e.double() - 10))


def nearest(a, table):
    """Index of the nearest of ascending values, ties to the even index; past the last: the last."""
    a = a.clamp(max=table[-1].item())
    hi = torch.bucketize(a, table).clamp(max=len(table) - 1)
    lo = (hi - 1).clamp(min=0)
    dl, dh = a - table[lo], table[hi] - a
    return torch.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)


def recipe(x):
    """Codes [rows][K], block scale codes [rows][K/16] and row scales of rows, each fp32 step made explicit."""
    x = x.double().cpu()
    rows, K = x.shape
    s = (x.abs().amax(1) / 2688).float()
    blocks, m = x.view(rows, -1, 16), x.view(rows, -1, 16).abs().amax(2)
    six = (s * 6).double()[:, None]
    b = nearest(torch.where(six > 0, m / six, 0.0).float().double(), e4m3_values())
    t = (e4m3_values()[b].float() * s[:, None]).double()[..., None]
    y = torch.where(t > 0, blocks / t, 0.0).float().double()
    c = nearest(y.abs(), SIZES) | (torch.signbit(y).long() << 3)
    return c.view(rows, K), b, s


def stored(c, b):
    """Codes two a byte and block scales in tiles of 128 rows and 4 blocks."""
    rows, K = c.shape
    q = (c[:, 0::2] | c[:, 1::2] << 4).to(torch.uint8)
    full = torch.zeros(-(-rows // 128) * 128, K // 16, dtype=torch.uint8)
    full[:rows] = b.to(torch.uint8)
    tiles = full.view(-1, 4, 32, K // 64, 4).permute(0, 3, 2, 1, 4).reshape(-1)
    return q, tiles


def written(rows, K):
    """Which bytes of the tiles belong to rows."""
    full = torch.zeros(-(-rows // 128) * 128, K // 16, dtype=torch.bool)
    full[:rows] = True
    return full.view(-1, 4, 32, K // 64, 4).permute(0, 3, 2, 1, 4).reshape(-1)


def values(c, b, s):
    """What the codes stand for: without the row scale, and with it as the recipe rounds it."""
    v = SIZES[c & 7] * (1 - 2 * (c >> 3)).double()
    blocks = v.view(*b.shape, 16)
    bare = (blocks * e4m3_values()[b][..., None]).view(c.shape)
    t = (e4m3_values()[b].float() * s[:, None]).double()
    return bare, (blocks * t[..., None]).view(c.shape)


def rows_of(rows, K, kind, seed=0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(rows, K, generator=g)
    if kind == "outliers":
        x[:, torch.randperm(K, generator=g)[: max(1, K // 50)]] *= 60
    if kind == "ranges":       # rows and blocks of any size, some of zeros
        x = x * torch.exp2(torch.randint(-40, 30, (rows, 1), generator=g).float())
        x = (x.view(rows, -1, 16) * torch.exp2(torch.randint(-14, 3, (rows, K // 16, 1), generator=g).float())).view(rows, K)
        x[::5] = 0
        x.view(rows, -1, 16)[1::3, ::2] = 0
    if kind == "ties":         # multiples of a quarter of the step, so that many quotients lie between codes
        x = torch.randint(-24, 25, (rows, K), generator=g).float() / 4
        x[:, 0] = 6.0
        x[1::2] *= 448
    if kind == "tiny":
        x = x * 2.0 ** -126
        x[0] = 2.0 ** -133
        x[-1] = 0
    return x


KINDS = ["plain", "outliers", "ranges", "ties", "tiny"]


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("rows,K", [(1, 64), (3, 128), (130, 320), (257, 1024), (40, 4096), (5, 16448), (2, 33024), (2, 65536)])
def test_rows(rows, K, kind):
    x = rows_of(rows, K, kind, seed=rows)
    for half in (True, False):
        src = x.to(torch.bfloat16) if half else x
        q, b, s = (moe.moe_quant_rows_fp4 if half else moe.moe_pack_fp4)(src.cuda())
        c, bb, ss = recipe(src)
        want_q, want_b = stored(c, bb)
        assert torch.equal(s.cpu(), ss)
        mine = written(rows, K)
        assert torch.equal(b.cpu()[mine], want_b[mine]) and (b.cpu()[~mine] == 0).all()
        assert torch.equal(q.cpu(), want_q)
        out = moe.moe_unpack_fp4(q, b, s)
        # (a code times its scales in fp32, then bf16: the product of 3 by 24 bits is rounded first)
        assert torch.equal(out.cpu(), values(c, bb, ss)[1].float().to(torch.bfloat16))


def test_every_code_comes_back():
    c = torch.arange(16).repeat(2, 4)
    b = torch.arange(8).view(2, 4) * 16 + 7
    s = torch.tensor([1.0, -0.37])
    q, tiles = stored(c, b)
    out = moe.moe_unpack_fp4(q.cuda(), tiles.cuda(), s.cuda())
    assert torch.equal(out.cpu(), values(c, b, s)[1].float().to(torch.bfloat16))


def project(x, w32, T, N, K, ws=None, out=None):
    q, b, s = moe.moe_pack_fp4(w32.cuda())
    ws = moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K)) if ws is None else ws
    out = torch.full((T, N), 7.0, dtype=torch.bfloat16, device="cuda") if out is None else out
    moe.moe_linear_fp4(x, moe.fp4(q, b, s), out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    return out


def check(out, x, w32):
    T, K = x.shape
    (xv, _), sx = values(*recipe(x)), recipe(x)[2]
    (wv, _), sw = values(*recipe(w32)), recipe(w32)[2]
    xv, wv = xv.cuda(), wv.cuda()
    scale = (sx.double()[:, None] * sw.double()).cuda()
    want = xv @ wv.T * scale
    size = xv.abs() @ wv.abs().T * scale
    # Products are exact.  A sum of K terms in fp32 that drops what lies below the accumulator's last bit is off by at most
    # K 2^-23 of the terms' sizes together; the two row scales round twice, bf16 once
    room = 2.0 ** -8 * want.abs() + (K + 8) * 2.0 ** -23 * size + 1e-37
    worst = ((out.double() - want).abs() / room).max().item()
    assert worst <= 1
    assert (out.double() - want).norm() <= 2.0 ** -8 * want.norm() + 1e-37


@pytest.mark.parametrize("T,N,K", [
    (1, 8, 64), (1, 256, 128), (2, 136, 192), (2, 8200, 4160), (2, 4096, 4096), (2, 6144, 4096), (256, 1024, 4096), (16, 16384, 1024), (1, 4104, 16448), (2, 72, 16448), (3, 1000, 448), (7, 128, 4096), (15, 520, 1024), (16, 256, 2048), (17, 264, 320), (31, 136, 576),
    (33, 384, 256), (64, 6144, 512), (100, 72, 1088), (127, 640, 640), (128, 128, 256), (129, 136, 64), (191, 1032, 832), (193, 256, 4160),
    (255, 504, 128), (257, 2048, 384), (500, 4096, 1024), (1000, 264, 8192), (2049, 1000, 320), (1, 40000, 64), (3, 8, 65536), (300, 8, 16448),
])
def test_projection(T, N, K):
    g = torch.Generator().manual_seed(T + N + K)
    x = rows_of(T, K, "outliers", seed=T).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g) / math.sqrt(K)
    check(project(x.cuda(), w, T, N, K), x, w)


# More wide tiles (128 tokens by 128 rows) than SMs: pairs of CTAs.  Halves of a tile without tokens or
# weight rows, K that ends inside a stage, one and several tiles to a pair.
@pytest.mark.parametrize("T,N,K", [
    (2049, 1400, 1088), (257, 10248, 1024), (300, 8200, 1984), (1100, 2568, 1344), (385, 16392, 4160), (2000, 1416, 1152), (20000, 136, 1024), (129, 20000, 1216), (2570, 1288, 64), (3000, 4104, 192),
])
def test_projection_by_pairs(T, N, K):
    g = torch.Generator().manual_seed(T + N + K)
    x = rows_of(T, K, "outliers", seed=T).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g) / math.sqrt(K)
    buf = torch.full((T + 130, N), 7.0, dtype=torch.bfloat16, device="cuda")
    check(project(x.cuda(), w, T, N, K, out=buf[:T]), x, w)
    assert (buf[T:] == 7).all()


# One and two tokens on either side of where the tensor cores take over.
@pytest.mark.parametrize("T,N,K", [
    (1, 9000, 4160), (1, 16384, 512), (1, 16392, 2048), (1, 33000, 448), (1, 8, 32768), (1, 8, 65536), (1, 6144, 8192), (2, 13000, 64), (2, 4104, 2048), (2, 1024, 8192),
    (2, 8, 16384), (2, 8, 16448), (2, 6152, 1984), (2, 1032, 16384),
])
def test_projection_of_one_and_two(T, N, K):
    g = torch.Generator().manual_seed(T + N + K)
    x = rows_of(T, K, "outliers", seed=T).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g) / math.sqrt(K)
    check(project(x.cuda(), w, T, N, K), x, w)


def test_pairs_captured_and_on_two_streams():
    T, N, K = 1300, 2056, 1088
    g = torch.Generator().manual_seed(8)
    xs = [torch.randn(T, K + 8, generator=g).to(torch.bfloat16).cuda()[:, :K] for _ in range(2)]
    w = torch.randn(N, K, generator=g)
    handle = moe.fp4(*moe.moe_pack_fp4(w.cuda()))
    want = [project(x, w, T, N, K) for x in xs]
    assert all(torch.equal(a, project(x.contiguous(), w, T, N, K)) for a, x in zip(want, xs))
    graphs = []
    for x in xs:
        graph, s, out = torch.cuda.CUDAGraph(), torch.cuda.Stream(), torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
        ws = moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K))
        with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
            moe.moe_linear_fp4(x, handle, out, ws)
        graphs.append((graph, s, out, ws))
    for _ in range(10):
        for graph, s, _, _ in graphs:
            with torch.cuda.stream(s):
                graph.replay()
    torch.cuda.synchronize()
    for (_, _, out, ws), a in zip(graphs, want):
        assert torch.equal(out, a) and moe.moe_check_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("T", [1, 40, 300])
def test_projection_of_any_rows(T, kind):
    N, K = 264, 704
    x, w = rows_of(T, K, kind, seed=1), rows_of(N, K, "plain" if kind == "tiny" else kind, seed=2)
    if kind in ("ranges", "ties"):
        x, w = x.clamp(-1e15, 1e15), w.clamp(-1e15, 1e15)
    x = x.to(torch.bfloat16)
    check(project(x.cuda(), w, T, N, K), x, w)


@pytest.mark.parametrize("T", [1, 33, 200])
def test_tokens_that_lie_apart(T):
    N, K = 256, 512
    wide = torch.randn(T, K + 72, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    w = torch.randn(N, K, generator=torch.Generator().manual_seed(2))
    x = wide[:, 8:8 + K]
    out = project(x, w, T, N, K)
    check(out, x.cpu(), w)
    assert torch.equal(out, project(x.contiguous(), w, T, N, K))


def test_a_workspace_serves_calls_of_any_sizes():
    g = torch.Generator().manual_seed(3)
    sizes = [(300, 512, 1024), (1, 6144, 4096), (17, 128, 64), (1, 6144, 4096), (129, 256, 4096), (2, 4096, 4096), (300, 512, 1024)]
    ws = moe.workspace(max(moe.moe_linear_fp4_workspace_bytes(*s) for s in sizes))
    first = {}
    for T, N, K in sizes:
        x = torch.randn(T, K, generator=torch.Generator().manual_seed(K)).to(torch.bfloat16)
        w = torch.randn(N, K, generator=torch.Generator().manual_seed(N))
        out = project(x.cuda(), w, T, N, K, ws)
        check(out, x, w)
        assert torch.equal(out, first.setdefault((T, N, K), out))
        assert torch.equal(out, project(x.cuda(), w, T, N, K))


def test_rows_behind_the_last_stay():
    T, N, K = 37, 200, 256
    x, w = torch.randn(T, K).to(torch.bfloat16), torch.randn(N, K)
    buf = torch.full((T + 200, N), 7.0, dtype=torch.bfloat16, device="cuda")
    project(x.cuda(), w, T, N, K, out=buf[:T])
    assert (buf[T:] == 7).all()
    check(buf[:T], x, w)


@pytest.mark.parametrize("T", [1, 20, 300])
def test_captured_calls_and_two_streams(T):
    N, K = 1024, 2048
    g = torch.Generator().manual_seed(T)
    xs = [torch.randn(T, K, generator=g).to(torch.bfloat16) for _ in range(3)]
    w = torch.randn(N, K, generator=g)
    packed = moe.moe_pack_fp4(w.cuda())
    handle = moe.fp4(*packed)
    want = [project(x.cuda(), w, T, N, K) for x in xs]
    x, ws = xs[0].cuda(), moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K))
    out = torch.zeros(T, N, dtype=torch.bfloat16, device="cuda")
    graph, s = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.stream(s), torch.cuda.graph(graph, stream=s):
        moe.moe_linear_fp4(x, handle, out, ws)
    for i in (1, 2, 0):
        x.copy_(xs[i])
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want[i])
    # two streams with a workspace each, at work at once
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K)) for _ in range(2)]
    outs = [[torch.zeros_like(out) for _ in range(10)] for _ in range(2)]
    xc = [v.cuda() for v in xs]
    torch.cuda.synchronize()
    for j in range(10):
        for i in range(2):
            moe.moe_linear_fp4(xc[i], handle, outs[i][j], spaces[i], stream=streams[i])
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(o, want[i]) for o in outs[i])


@pytest.mark.parametrize("T,N,K", [(40, 512, 4096), (20, 8192, 1024), (300, 512, 4096), (3000, 2048, 1024), (600, 4096, 512)])
@pytest.mark.parametrize("stage", [1, 2])   # (a CTA of eight that share 16 stages has two)
def test_a_wait_that_runs_out(T, N, K, stage):
    """CTA 0 skips the copies of one stage: the call ends with the status, and the workspace serves the next call."""
    x = torch.randn(T, K, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).cuda()
    w = moe.fp4(*moe.moe_pack_fp4(torch.randn(N, K, generator=torch.Generator().manual_seed(2)).cuda()))
    ws = moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K))
    out, want = (torch.zeros(T, N, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    moe.moe_linear_fp4(x, w, want, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    moe.moe_debug_set_waits(ws, 1_000_000, stage)     # 1 ms: every other wait of these launches takes microseconds
    moe.moe_linear_fp4(x, w, out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    moe.moe_debug_set_waits(ws, 0, 0)
    moe.moe_linear_fp4(x, w, out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK and torch.equal(out, want)


def test_empty_calls():
    w = moe.fp4(*moe.moe_pack_fp4(torch.randn(64, 128, device="cuda")))
    x, out = torch.empty(0, 128, dtype=torch.bfloat16, device="cuda"), torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear_fp4(x, w, out, moe.workspace(256))
    q, b, s = moe.moe_quant_rows_fp4(x)
    assert q.shape == (0, 64) and b.numel() == 0 and s.numel() == 0


def test_the_binding_refuses():
    T, N, K = 4, 64, 128
    x, w = torch.randn(T, K, device="cuda").to(torch.bfloat16), moe.moe_pack_fp4(torch.randn(N, K, device="cuda"))
    h, out = moe.fp4(*w), torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    ws = moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K))
    for args in ((x[:, :64], h, out), (x, h, out[:3]), (x.half(), h, out), (x.float(), h, out), (x.cpu(), h, out), (x, h, out.cpu()),
                 (x, moe.Fp4(), out), (x.t(), h, out)):
        with pytest.raises(ValueError):
            moe.moe_linear_fp4(*args, ws)
    with pytest.raises(ValueError):
        moe.fp4(w[0], w[1][:-1], w[2])
    with pytest.raises(ValueError):
        moe.moe_quant_rows_fp4(x, w[0])
    with pytest.raises(moe.MoeError):
        moe.moe_linear_fp4(x, h, out, ws[:256])
    with pytest.raises(moe.MoeError):
        moe.moe_pack_fp4(torch.randn(4, 96, device="cuda"))
