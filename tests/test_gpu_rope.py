"""Rotary positions: tables against 64 bits, rows against the same steps in fp32 on the CPU (bit for bit where no
norm's sum comes first), and keys and values in the cache against their recipe."""
import math

import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from attn_cases import FORMATS, quantise, slots_view

pytestmark = pytest.mark.gpu


def frequencies(g):
    """Each pair's angle per position, by the formulas one by one."""
    f = []
    for i in range(g.rot // 2):
        w = g.base ** (-2.0 * i / g.rot)
        keep = 1.0
        if g.scaling == moe.MOE_ROPE_LINEAR:
            keep = 0.0
        if g.scaling == moe.MOE_ROPE_RAMP:
            pair = lambda t: g.rot * math.log(g.orig_len / (2 * math.pi * t)) / (2 * math.log(g.base))  # noqa: E731
            a, b = max(math.floor(pair(g.hi)), 0), min(math.ceil(pair(g.lo)), g.rot - 1)
            keep = 1 - min(max((i - a) / max(b - a, 0.001), 0), 1)
        if g.scaling == moe.MOE_ROPE_BAND:
            keep = min(max((g.orig_len * w / (2 * math.pi) - g.lo) / (g.hi - g.lo), 0), 1)
        f.append(w * keep + (1 - keep) * w / g.factor if keep else w / g.factor)
    return torch.tensor(f, dtype=torch.float64)


def config(**kw):
    base = dict(base=10000.0, factor=8.0, orig_len=4096.0, lo=1.0, hi=32.0, magnitude=1.0, rot=64, scaling=0)
    base.update(kw)
    return moe.RopeConfig(**base)


@pytest.mark.parametrize("kw,pos0,n", [
    (dict(), 0, 1), (dict(rot=16), 0, 1000), (dict(rot=128, base=5e5), 131000, 300), (dict(rot=256), (1 << 24) - 100, 100),
    (dict(scaling=1), 7, 500), (dict(scaling=2, rot=128, magnitude=1.2079), 60000, 333),
    (dict(scaling=3, rot=96, lo=1.0, hi=4.0, base=5e5), 100000, 257), (dict(scaling=2, orig_len=3.0), 0, 50),
    (dict(scaling=1, factor=1.0), 0, 100), (dict(base=1.0000001), 12345, 65),
])
def test_table(kw, pos0, n):
    g = config(**kw)
    table = torch.full((n, g.rot), 7.0, device="cuda")
    moe.moe_rope_table(g, pos0, table)
    a = torch.arange(pos0, pos0 + n, dtype=torch.float64)[:, None] * frequencies(g)
    want = torch.cat((a.cos(), a.sin()), 1) * g.magnitude
    # the reduced angle in 24 bits and one unit of each function (2^-24 each at most), the factor's
    # rounding, and the 53 bits of the frequency times up to 2^24 on either side: below 2^-22 in all
    assert (table.cpu().double() - want).abs().max() <= 2.0 ** -22 * g.magnitude


def test_table_ends_at_the_last_position():
    g = config(rot=16, base=1e6)
    table = torch.full((2, 16), 7.0, device="cuda")
    moe.moe_rope_table(g, 2**31 - 2, table)
    f = frequencies(g)
    a = torch.tensor([2.0**31 - 2, 2.0**31 - 1], dtype=torch.float64)[:, None] * f
    # 2^31 times a frequency of 53 bits (a few units off on either side): 2^-19 of an angle
    assert (table.cpu().double() - torch.cat((a.cos(), a.sin()), 1)).abs().max() <= 2.0 ** -19


def test_far_tables_repeat_nothing():
    # rows of a table made in one call are those made in pieces
    g = config(rot=128, scaling=2)
    whole, part = torch.empty(1000, 128, device="cuda"), torch.empty(400, 128, device="cuda")
    moe.moe_rope_table(g, 5000, whole)
    moe.moe_rope_table(g, 5300, part)
    assert torch.equal(whole[300:700], part)


def rotated(x, w, eps, row, rot, pairs, inverse=False, dtype=torch.float32):
    """Rows [T][H][D], step by step in the given type."""
    x = x.to(dtype)
    if w is not None:
        x = x * torch.rsqrt(x.square().mean(-1, keepdim=True) + eps) * w.to(dtype)
    c, s = row[:, None, : rot // 2].to(dtype), row[:, None, rot // 2:].to(dtype)
    if inverse:
        s = -s
    p = x[..., :rot]
    a, b = (p[..., 0::2], p[..., 1::2]) if pairs else (p[..., : rot // 2], p[..., rot // 2:])
    u, v = a * c - b * s, b * c + a * s
    y = torch.stack((u, v), -1).flatten(-2) if pairs else torch.cat((u, v), -1)
    return torch.cat((y, x[..., rot:]), -1)


def table_of(n, rot):
    t = torch.empty(n, rot, device="cuda")
    moe.moe_rope_table(config(rot=rot), 0, t)
    return t


def bf16_close(got, want, terms=0):
    """A bf16 rounding of the exact value (half a step, 2^-8 relative), and fp32 steps before it."""
    got, want = got.double().cpu(), want.double().cpu()
    over = ((got - want).abs() - 2.0 ** -8 * want.abs()).max().item()
    assert over <= terms


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [
    (1, 1, 64, 16), (1, 32, 128, 128), (3, 5, 64, 64), (17, 7, 128, 48), (700, 2, 128, 64), (5000, 9, 64, 32), (40, 130, 128, 112),
    (20001, 8, 128, 128),
])
def test_rows(T, H, D, rot, pairs):
    g = torch.Generator().manual_seed(T + rot)
    wide = torch.randn(T, H * D + 24, generator=g).to(torch.bfloat16).cuda()
    x = wide[:, 8:8 + H * D].view(T, H, D)
    table = table_of(3000, rot)
    pos = torch.randint(0, 3000, (T,), generator=g).to(torch.int32).cuda()
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    ws = moe.workspace(256)
    flags = moe.MOE_ROPE_PAIRS if pairs else 0
    moe.moe_rope_rows(x, pos, moe.rope(table, flags), out, ws)
    row = table[pos.long()]
    want = rotated(x, None, 0, row, rot, pairs).to(torch.bfloat16)
    assert torch.equal(out.view(torch.int16), want.view(torch.int16))
    # in place, on a slice: nothing beside it changes
    moe.moe_rope_rows(x, pos, moe.rope(table, flags), x, ws)
    assert torch.equal(x, want)
    assert torch.equal(wide[:, :8].cpu(), torch.randn(T, H * D + 24, generator=torch.Generator().manual_seed(T + rot))[:, :8].to(torch.bfloat16))
    assert moe.moe_check_device_status(ws) == moe.MOE_OK


@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H,D,rot", [(1, 3, 64, 32), (9, 8, 128, 128), (300, 5, 128, 16)])
def test_rows_with_a_norm(T, H, D, rot, pairs):
    g = torch.Generator().manual_seed(3)
    x = (torch.randn(T, H, D, generator=g) * torch.logspace(-6, 6, T)[:, None, None]).to(torch.bfloat16)
    x[-1, 0] = 0
    w = torch.randn(D, generator=g)
    table = table_of(100, rot)
    pos = torch.randint(0, 100, (T,), generator=g)
    out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_rope_rows(x.cuda(), pos.to(torch.int32).cuda(),
                      moe.rope(table, moe.MOE_ROPE_PAIRS if pairs else 0, q_norm=w.cuda(), eps=1e-6), out, moe.workspace(256))
    want = rotated(x, w, 1e-6, table.cpu()[pos], rot, pairs, dtype=torch.float64)
    # fp32 before the rounding: the sum of squares is off by D 2^-24 at most, half of it in the root, products and
    # the pair's sum by some units: below 2^-17 of the pair's two terms, |x w / rms| <= sqrt(D) |w|
    bf16_close(out, want, 2.0 ** -17 * 2 * math.sqrt(D) * w.abs().max().item())


@pytest.mark.parametrize("pairs", [False, True])
def test_inverse_is_the_gradient(pairs):
    T, H, D, rot = 50, 3, 64, 48
    g = torch.Generator().manual_seed(4)
    table, pos = table_of(1000, rot), torch.randint(0, 1000, (T,), generator=g).to(torch.int32).cuda()
    x, dy = (torch.randn(T, H, D, generator=g).to(torch.bfloat16).cuda() for _ in range(2))
    flags, ws = moe.MOE_ROPE_PAIRS if pairs else 0, moe.workspace(256)
    dx = torch.empty_like(dy)
    moe.moe_rope_rows(dy, pos, moe.rope(table, flags | moe.MOE_ROPE_INVERSE), dx, ws)
    # the gradient that automatic differentiation gives of the formula
    leaf = x.double().cpu().requires_grad_()
    rotated(leaf, None, 0, table[pos.long()].cpu(), rot, pairs, dtype=torch.float64).backward(dy.double().cpu())
    bf16_close(dx, leaf.grad, 2.0 ** -22 * 8)
    # and its differences: the map is linear, so one element moved by 1 in each head shows its column
    at = torch.randint(0, D, (T, H, 1), generator=g).cuda()
    e = torch.zeros_like(x).scatter_(2, at, 1.0)
    y = [torch.empty_like(x) for _ in range(2)]
    moe.moe_rope_rows(e, pos, moe.rope(table, flags), y[0], ws)
    terms = y[0].double() * dy.double()
    moved, want = terms.sum(-1), dx.gather(2, at).double().squeeze(-1)
    assert ((moved - want).abs() <= 2.0 ** -8 * (terms.abs().sum(-1) + want.abs()) + 2.0 ** -20).all()
    moe.moe_rope_rows(x, pos, moe.rope(table, flags), y[0], ws)
    # and back again
    moe.moe_rope_rows(y[0], pos, moe.rope(table, flags | moe.MOE_ROPE_INVERSE), y[1], ws)
    assert (y[1].double() - x.double()).abs().max() <= 2.0 ** -7 * 8


def test_tokens_left_out():
    T, H, D = 6, 2, 64
    x = torch.randn(T, H, D, device="cuda").to(torch.bfloat16)
    table = table_of(10, 64)
    pos = torch.tensor([0, -1, 9, 10, -(1 << 31), (1 << 31) - 1], dtype=torch.int32, device="cuda")
    out = torch.full_like(x, 7.0)
    ws = moe.workspace(256)
    moe.moe_rope_rows(x, pos, moe.rope(table), out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert torch.equal(out[0], x[0])
    assert (out[[1, 3, 4, 5]] == 7).all() and not (out[2] == 7).any()
    moe.moe_rope_rows(x[:2], pos[:2], moe.rope(table), out[:2], ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK


def _write_setup(T, H, H_kv, D, page, fmt, layout, seed=0, spare=40):
    g = torch.Generator().manual_seed(seed)
    n_pages = -(-T // page) + spare // page + 1
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    qkv = torch.randn(T, (H + 2 * H_kv) * D + 8, generator=g).to(torch.bfloat16).cuda()
    q = qkv[:, :H * D].view(T, H, D)
    k = qkv[:, H * D:(H + H_kv) * D].view(T, H_kv, D)
    v = qkv[:, (H + H_kv) * D:(H + 2 * H_kv) * D].view(T, H_kv, D)
    row = D // 2 if fmt == "int4" else D
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    pool = [slots_view(torch.full((n_pages, H_kv, page, row), 3, dtype=dt, device="cuda"), layout) for _ in range(2)]
    sc = [torch.full((n_pages, H_kv, page), 5.0, device="cuda") if fmt != "bf16" else None for _ in range(2)]
    dims = moe.KvDims(T=T, B=1, H=H, H_kv=H_kv, D=D, page=page, n_pages=n_pages, max_pages=n_pages, max_new=0, window=0,
                      format=FORMATS.index(fmt), flags=0)
    pos = torch.randint(0, 2000, (T,), generator=g).to(torch.int32)
    return q, k, v, slots, pos, pool, sc, dims, moe.kv_cache(*pool, *sc)


def codes_of(x, fmt):
    """The recipe on fp32 rows, on the CPU: stored codes and scales."""
    x = x.cpu()
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    return tuple(t.cuda() for t in quantise(x, fmt))


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("pairs", [False, True])
@pytest.mark.parametrize("T,H,H_kv,D,rot,page,layout", [
    (1, 1, 1, 64, 64, 16, "heads"), (1, 32, 8, 128, 128, 16, "heads"), (5, 14, 2, 64, 32, 32, "tokens"),
    (301, 6, 3, 128, 48, 64, "strided"), (3000, 8, 8, 128, 64, 128, "tokens"), (9000, 20, 4, 64, 16, 256, "heads"),
])
def test_write(T, H, H_kv, D, rot, page, layout, pairs, fmt):
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(T, H, H_kv, D, page, fmt, layout)
    pos[T // 3::7] = -1            # padding, and tokens whose key and value are not wanted
    slots[T // 2::5] = -1
    pos, slots = pos.cuda(), slots.cuda()
    table, ws = table_of(2000, rot), moe.workspace(256)
    out = torch.full((T, H, D), 7.0, dtype=torch.bfloat16, device="cuda")
    before = [None if t is None else t.clone() for t in (*pool, *sc)]
    moe.moe_rope_kv_write(q, k, v, pos, slots, moe.rope(table, moe.MOE_ROPE_PAIRS if pairs else 0), dims, cache, out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    row = table[pos.clamp(min=0).long()]
    want = rotated(q, None, 0, row, rot, pairs).to(torch.bfloat16)
    want[pos < 0] = 7.0
    assert torch.equal(out, want)
    live = (pos >= 0) & (slots >= 0)
    p, at = slots[live].long() // page, slots[live].long() % page
    turned = rotated(k, None, 0, row, rot, pairs)
    for x, rows, s, was, was_s in ((turned, pool[0], sc[0], before[0], before[2]), (v.float(), pool[1], sc[1], before[1], before[3])):
        codes, scales = codes_of(x[live], fmt)
        was[p, :, at] = codes.cuda()
        assert torch.equal(rows, was)
        if s is not None:
            was_s[p, :, at] = scales
            assert torch.equal(s, was_s)


@pytest.mark.parametrize("T", [1, 130, 4000])
def test_write_is_rows_and_write(T):
    """In bf16, with norms, the fused call gives what the single ones give."""
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(T, 12, 4, 128, 16, "bf16", "heads")
    pos, slots = pos.cuda(), slots.cuda()
    w = [torch.randn(128, device="cuda") for _ in range(2)]
    table, ws = table_of(2000, 96), moe.workspace(256)
    out, out2, kr = torch.empty(T, 12, 128, dtype=torch.bfloat16, device="cuda"), *(torch.empty(T, h, 128, dtype=torch.bfloat16, device="cuda") for h in (12, 4))
    moe.moe_rope_rows(q, pos, moe.rope(table, 0, q_norm=w[0], eps=1e-5), out2, ws)
    moe.moe_rope_rows(k, pos, moe.rope(table, 0, q_norm=w[1], eps=1e-5), kr, ws)
    moe.moe_kv_write(kr, v, slots, dims, cache, ws)
    want = [t.clone() for t in pool]
    for t in pool:
        t.fill_(3)
    moe.moe_rope_kv_write(q, k, v, pos, slots, moe.rope(table, 0, *w, 1e-5), dims, cache, out, ws)
    assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(pool, want))


@pytest.mark.parametrize("fmt", FORMATS)
def test_write_with_norms(fmt):
    T, H, H_kv, D, rot, page = 77, 6, 2, 128, 64, 16
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(T, H, H_kv, D, page, fmt, "heads")
    w = [torch.randn(D) for _ in range(2)]
    table, ws = table_of(2000, rot), moe.workspace(256)
    out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_rope_kv_write(q, k, v, pos.cuda(), slots.cuda(), moe.rope(table, 0, w[0].cuda(), w[1].cuda(), 1e-6), dims, cache, out, ws)
    back = torch.empty(2, T, H_kv, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_read(slots.cuda(), dims, cache, back[0], back[1], ws)
    row = table.cpu()[pos.long()]
    room = 2.0 ** -17 * 2 * math.sqrt(D)
    bf16_close(out, rotated(q.cpu(), w[0], 1e-6, row, rot, False, dtype=torch.float64), room * w[0].abs().max().item())
    want = rotated(k.cpu(), w[1], 1e-6, row, rot, False, dtype=torch.float64)
    room *= w[1].abs().max().item()
    got, top = back[0].double().cpu(), want.abs().amax(-1, keepdim=True)
    # half a code step (E4M3: 2^-4 of the value or of the smallest normal's step, int4: absmax / 14), the reading's bf16
    step = {"bf16": 0 * top, "e4m3": torch.maximum(want.abs() * 2.0 ** -4, top / 448 * 2.0 ** -10), "int4": top / 14}[fmt]
    assert ((got - want).abs() <= step * (1 + 2.0 ** -8) + 2.0 ** -8 * want.abs() + 2 * room).all()


def test_bad_slots_and_positions():
    T = 5
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(T, 4, 2, 64, 16, "e4m3", "heads")
    table, ws = table_of(2000, 64), moe.workspace(256)
    was = [t.clone() for t in (*pool, *sc)]
    out = torch.full((T, 4, 64), 7.0, dtype=torch.bfloat16, device="cuda")
    n = dims.n_pages * dims.page
    moe.moe_rope_kv_write(q, k, v, torch.full((T,), 2000, dtype=torch.int32, device="cuda"), slots.cuda(), moe.rope(table), dims, cache, out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert (out == 7).all()
    moe.moe_rope_kv_write(q, k, v, pos.cuda(), torch.full((T,), n, dtype=torch.int32, device="cuda"), moe.rope(table), dims, cache, out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert torch.equal(out, rotated(q, None, 0, table[pos.cuda().long()], 64, False).to(torch.bfloat16))
    assert all(torch.equal(a, b) for a, b in zip((*pool, *sc), was))


def test_rows_of_zeros_and_their_scales():
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(3, 2, 1, 64, 16, "int4", "heads")
    k.zero_()
    v.zero_()
    table, ws = table_of(2000, 64), moe.workspace(256)
    out = torch.empty(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    moe.moe_rope_kv_write(q, k, v, pos.cuda(), slots.cuda(), moe.rope(table), dims, cache, out, ws)
    back = torch.full((2, 3, 1, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_read(slots.cuda(), dims, cache, back[0], back[1], ws)
    assert (back == 0).all()


def test_the_binding_refuses():
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(4, 4, 2, 64, 16, "e4m3", "heads")
    pos, slots, table, ws = pos.cuda(), slots.cuda(), table_of(2000, 64), moe.workspace(256)
    out, r = torch.empty(4, 4, 64, dtype=torch.bfloat16, device="cuda"), moe.rope(table)
    bad_norm = moe.rope(table, 0, torch.ones(128, device="cuda"))
    for args in ((q, k, v, pos, slots, bad_norm, dims, cache, out), (q[:3], k, v, pos, slots, r, dims, cache, out),
                 (q, q, v, pos, slots, r, dims, cache, out), (q, k, v, pos[:3], slots, r, dims, cache, out),
                 (q.half(), k, v, pos, slots, r, dims, cache, out), (q, k, v, pos, slots.long(), r, dims, cache, out),
                 (q, k, v, pos, slots, r, dims, cache, out.cpu()), (q, k, v, pos, slots, r, dims.replace(page=32), cache, out)):
        with pytest.raises(ValueError):
            moe.moe_rope_kv_write(*args, ws)
    with pytest.raises(ValueError):
        moe.rope(table, 0, torch.ones(64, device="cuda"), torch.ones(128, device="cuda"))
    with pytest.raises(ValueError):
        moe.moe_rope_table(config(rot=32), 0, table)
    with pytest.raises(moe.MoeError):
        moe.moe_rope_rows(q, pos, moe.rope(table, 8), out, ws)
