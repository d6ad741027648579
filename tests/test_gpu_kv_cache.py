"""Writing the paged cache and reading it back: codes, scales and values equal to the recipe in
64 bits, bit for bit."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from attn_cases import FORMATS, quantise, slots_view, values

pytestmark = pytest.mark.gpu


def _setup(T, H_kv, D, page, fmt, layout="heads", pad=0, seed=0, spare=40, gain=1.0):
    g = torch.Generator().manual_seed(seed)
    n_pages = -(-T // page) + spare // page + 1
    slots = torch.randperm(n_pages * page, generator=g)[:T].to(torch.int32)
    slots[T - pad:] = -1
    wide = (torch.randn((T, 2 * H_kv * D + 8), generator=g) * gain).to(torch.bfloat16).cuda()
    k = wide[:, :H_kv * D].view(T, H_kv, D)
    v = wide[:, H_kv * D:2 * H_kv * D].view(T, H_kv, D)
    row = D // 2 if fmt == "int4" else D
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    pool = [slots_view(torch.full((n_pages, H_kv, page, row), 3, dtype=dt, device="cuda"), layout)
            for _ in range(2)]
    sc = [torch.full((n_pages, H_kv, page), 5.0, device="cuda") if fmt != "bf16" else None
          for _ in range(2)]
    dims = moe.KvDims(T=T, B=1, H=H_kv, H_kv=H_kv, D=D, page=page, n_pages=n_pages,
                      max_pages=n_pages, max_new=0, window=0, format=FORMATS.index(fmt), flags=0)
    return k, v, slots.cuda(), pool, sc, dims, moe.kv_cache(*pool, *sc), moe.workspace(256)


def _check(k, v, slots, pool, sc, page, fmt, before):
    live = slots >= 0
    p, at = slots[live].long() // page, slots[live].long() % page
    for x, rows, s, was in ((k, pool[0], sc[0], before[0]), (v, pool[1], sc[1], before[1])):
        codes, scales = quantise(x[live], fmt)
        want = was.clone()
        want[p, :, at] = codes
        assert torch.equal(rows.view(torch.int16) if fmt == "bf16" else rows,
                           want.view(torch.int16) if fmt == "bf16" else want)
        if s is not None:
            ws = torch.full_like(s, 5.0)
            ws[p, :, at] = scales
            assert torch.equal(s, ws)


def _back(k, fmt):
    codes, s = quantise(k, fmt)
    return values(codes, s, fmt).float().to(torch.bfloat16)


@pytest.mark.parametrize("fmt", FORMATS)
@pytest.mark.parametrize("T,H_kv,D,page,layout,pad", [
    (1, 1, 64, 16, "heads", 0), (1, 8, 128, 16, "heads", 0), (3, 5, 64, 32, "tokens", 1),
    (257, 3, 128, 64, "strided", 17), (1000, 8, 128, 128, "tokens", 0), (129, 1, 64, 256, "heads", 129),
])
def test_write_and_read_back(fmt, T, H_kv, D, page, layout, pad):
    k, v, slots, pool, sc, dims, cache, ws = _setup(T, H_kv, D, page, fmt, layout, pad)
    before = [p.clone() for p in pool]
    moe.moe_kv_write(k, v, slots, dims, cache, ws)
    ko, vo = torch.full((2, T, H_kv, D), 9.0, dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_read(slots, dims, cache, ko, vo, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    _check(k, v, slots, pool, sc, page, fmt, before)
    live = slots >= 0
    for got, x in ((ko, k), (vo, v)):
        assert torch.equal(got[live], _back(x[live], fmt))
        assert (got[~live] == 0).all()


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
def test_rows_at_the_edges_of_the_formats(fmt):
    """All-zero rows, one large element, halves between codes, the smallest and largest bf16."""
    T, H_kv, D, page = 8, 1, 128, 16
    k, v, slots, pool, sc, dims, cache, ws = _setup(T, H_kv, D, page, fmt)
    k = k.contiguous()
    k[0] = 0
    k[1] = 0
    k[1, 0, 77] = -3.0e38
    k[2, 0] = torch.arange(-64, 64).to(torch.bfloat16) / 8            # ties of int4 at absmax 7, 8
    k[3, 0] = torch.linspace(-448, 448, D).to(torch.bfloat16)
    k[4, 0] = 2.0 ** -126
    k[5, 0] = torch.linspace(-7, 7, D).to(torch.bfloat16)
    k[6, 0] = -k[2, 0]
    k[7, 0, ::2] = 0.0
    k[7, 0, 1::4] = -0.0
    v = v.contiguous()
    before = [p.clone() for p in pool]
    moe.moe_kv_write(k, v, slots, dims, cache, ws)
    ko, vo = torch.empty((2, T, H_kv, D), dtype=torch.bfloat16, device="cuda")
    moe.moe_kv_read(slots, dims, cache, ko, vo, ws)
    got, want = pool[0].clone(), before[0].clone()
    codes, scales = quantise(k, fmt)
    p, at = slots.long() // page, slots.long() % page
    want[p, :, at] = codes
    zero_row = got[p[0], :, at[0]]
    assert (zero_row == 0).all() and sc[0][p[0], 0, at[0]] == 0
    assert torch.equal(got, want)
    assert torch.equal(ko, _back(k, fmt))


@pytest.mark.parametrize("fmt", ["e4m3", "int4"])
@pytest.mark.parametrize("power", [0, 100, -60, -110, -125])
def test_quotients_of_every_pair_of_significands(fmt, power):
    """Each of the 128 bf16 significands under each maximum, over the codes' whole range (most
    midpoints between codes that bf16 rows can meet are among them), at ordinary scales and at the largest
    and smallest."""
    D, H_kv = 128, 8
    sig = (128 + torch.arange(128)).double()
    rows = []
    for top in range(128):
        for e in range(8):      # elements a factor 2^-e (and up to 2^-1 more) below the maximum
            x = sig * 2.0 ** -e
            x[x > sig[top]] /= 2
            x[::2] *= -1
            x[0] = sig[top]
            rows.append(x * 2.0 ** (power - 7))
    k = torch.stack(rows).to(torch.bfloat16).view(128, H_kv, D).cuda()
    T = k.shape[0]
    _, _, slots, pool, sc, dims, cache, ws = _setup(T, H_kv, D, 64, fmt)
    v = -k
    moe.moe_kv_write(k, v, slots, dims, cache, ws)
    p, at = slots.long() // 64, slots.long() % 64
    for x, rows, s in ((k, pool[0], sc[0]), (v, pool[1], sc[1])):
        codes, scales = quantise(x, fmt)
        assert torch.equal(s[p, :, at], scales)
        assert torch.equal(rows[p, :, at], codes)


@pytest.mark.parametrize("fmt", ["bf16", "int4"])
def test_slots_past_the_pool(fmt):
    """Not written, read as zeros, and recorded; the other rows are as ever."""
    k, v, slots, pool, sc, dims, cache, ws = _setup(20, 2, 64, 16, fmt)
    bad = slots.clone()
    bad[3], bad[11] = dims.n_pages * 16, 2 ** 31 - 1
    before = [p.clone() for p in pool]
    moe.moe_kv_write(k, v, bad, dims, cache, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    bad[3] = bad[11] = -1
    _check(k, v, bad, pool, sc, 16, fmt, before)
    ko, vo = torch.full((2, 20, 2, 64), 9.0, dtype=torch.bfloat16, device="cuda")
    slots[5] = dims.n_pages * 16
    moe.moe_kv_read(slots, dims, cache, ko, vo, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    assert (ko[5] == 0).all() and (vo[5] == 0).all()
    assert torch.equal(vo[7], _back(v[7], fmt))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3"])
def test_pool_past_32_bits(fmt):
    """Rows whose byte (and, for bf16, element) offsets pass 2^32."""
    H_kv, D, page = 8, 128, 256
    size = 2 if fmt == "bf16" else 1
    n_pages = (1 << 33) // (H_kv * D * page * 2) + 3 if fmt == "bf16" else (1 << 32) // (H_kv * D * page) + 3
    dt = torch.bfloat16 if fmt == "bf16" else torch.uint8
    k_pool, v_pool = (torch.empty((n_pages, H_kv, page, D), dtype=dt, device="cuda") for _ in range(2))
    ks, vs = ((None, None) if fmt == "bf16" else
              (torch.empty((n_pages, H_kv, page), device="cuda") for _ in range(2)))
    T = 5
    dims = moe.KvDims(T=T, B=1, H=8, H_kv=8, D=D, page=page, n_pages=n_pages, max_pages=1,
                      max_new=0, window=0, format=FORMATS.index(fmt), flags=0)
    assert n_pages * H_kv * page * D * size > 1 << 32
    slots = torch.tensor([0, n_pages * page - 1, n_pages * page - 255, 7, (n_pages - 2) * page],
                         dtype=torch.int32, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(3)
    k, v = torch.randn((2, T, 8, D), generator=g, device="cuda").to(torch.bfloat16)
    ws = moe.workspace(256)
    cache = moe.kv_cache(k_pool, v_pool, ks, vs)
    moe.moe_kv_write(k, v, slots, dims, cache, ws)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    moe.moe_kv_read(slots, dims, cache, ko, vo, ws)
    assert torch.equal(ko, _back(k, fmt)) and torch.equal(vo, _back(v, fmt))
    p, at = slots.long() // page, slots.long() % page
    assert torch.equal(k_pool[p, :, at].view(torch.uint8), quantise(k, fmt)[0].view(torch.uint8))


def test_other_stream_and_graph():
    """The calls run on the stream they are given, and again from a captured graph."""
    k, v, slots, pool, sc, dims, cache, ws = _setup(40, 2, 128, 16, "e4m3")
    ko, vo = torch.zeros((2, 40, 2, 128), dtype=torch.bfloat16, device="cuda")
    torch.cuda.synchronize()
    st = torch.cuda.Stream()
    moe.moe_kv_write(k, v, slots, dims, cache, ws, stream=st)
    moe.moe_kv_read(slots, dims, cache, ko, vo, ws, stream=st)
    st.synchronize()
    assert torch.equal(ko, _back(k, "e4m3"))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        moe.moe_kv_write(k, v, slots, dims, cache, ws)
        moe.moe_kv_read(slots, dims, cache, ko, vo, ws)
    k.mul_(2.0)
    ko.zero_()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(ko, _back(k, "e4m3"))


def test_binding_refuses():
    k, v, slots, pool, sc, dims, cache, ws = _setup(20, 2, 64, 16, "int4")
    for bad in (lambda: moe.moe_kv_write(k[:19], v, slots, dims, cache, ws),
                lambda: moe.moe_kv_write(k, v, slots[:19], dims, cache, ws),
                lambda: moe.moe_kv_write(k, v, slots.long(), dims, cache, ws),
                lambda: moe.moe_kv_write(k.float(), v, slots, dims, cache, ws),
                lambda: moe.moe_kv_write(k, v, slots, dims.replace(D=128), cache, ws),
                lambda: moe.moe_kv_write(k, v, slots, dims.replace(format=1), cache, ws),
                lambda: moe.kv_cache(pool[0], pool[1]),
                lambda: moe.kv_cache(pool[0], pool[1], sc[0], sc[1][:, :1]),
                lambda: moe.kv_cache(pool[0], pool[1].permute(0, 2, 1, 3), *sc),
                lambda: moe.moe_kv_read(slots, dims, cache, k, k[:3], ws)):
        with pytest.raises(ValueError):
            bad()
    with pytest.raises(moe.MoeError):
        moe.moe_kv_write(k, v, slots, dims, cache, ws[:128])
