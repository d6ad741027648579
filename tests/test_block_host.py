"""Refusals of page planning, rotary positions, block norms and 4-bit floats: every bad argument comes back
as its documented status (or a ValueError of the binding) before anything is enqueued."""
import ctypes
import math

import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

INV, UNS, WS, OK_ = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE, moe.MOE_OK
OK, BAD, ODD = 1 << 21, (1 << 21) + 8, (1 << 21) + 2     # addresses, never dereferenced


@pytest.fixture(scope="module")
def L():
    import moe_expert_layer_sigmoid_gb300.build as b
    b.build()
    return moe.lib()


def _dims(**kw):
    base = dict(T=4, B=2, H=8, H_kv=2, D=128, page=16, n_pages=10, max_pages=4, max_new=0, window=0,
                format=moe.MOE_KV_E4M3, flags=0)
    base.update(kw)
    return moe.KvDims(**base)


def _plan(L, d=None, new=OK, st=None, off=OK, pos=OK, slots=OK, ws=1 << 20, n=256, **state):
    held = dict(kv_len=OK, first=OK, pages=OK, free_pages=OK, n_free=OK)
    held.update(state)
    return L.moe_kv_plan(new, ctypes.byref(d or _dims()), ctypes.byref(st or moe.KvPages(**held)), off, pos, slots,
                         ws, n, None)


def _rope(**kw):
    base = dict(table=OK, q_norm=None, k_norm=None, n_pos=100, rot=64, flags=0, eps=0.0)
    base.update(kw)
    return moe.Rope(**base)


def _cache(**kw):
    base = dict(k=OK, v=OK, ks=OK, vs=OK, page_stride=4096, head_stride=2048, slot_stride=128)
    base.update(kw)
    return moe.Kv(**base)


def _rows(L, r=None, x=OK, ldx=1024, pos=OK, T=4, H=8, D=128, out=OK + 4096, ldo=1024, ws=1 << 20, n=256):
    return L.moe_rope_rows(x, ldx, pos, T, H, D, ctypes.byref(r or _rope()), out, ldo, ws, n, None)


def _write(L, d=None, r=None, c=None, q=OK, ldq=1024, k=OK, ldk=256, v=OK, ldv=256, pos=OK, slots=OK, out=OK + 4096,
           ldo=1024, ws=1 << 20, n=256):
    return L.moe_rope_kv_write(q, ldq, k, ldk, v, ldv, pos, slots, ctypes.byref(r or _rope()),
                               ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), out, ldo, ws, n, None)


DIMS = [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(H=0), INV), (dict(H_kv=0), INV), (dict(H=7), INV), (dict(page=0), INV),
    (dict(n_pages=0), INV), (dict(max_pages=0), INV), (dict(window=-1), INV), (dict(flags=1), INV), (dict(D=96), UNS),
    (dict(page=8), UNS), (dict(page=48), UNS), (dict(format=3), UNS), (dict(B=8193), UNS), (dict(n_pages=1 << 27), UNS),
    (dict(max_pages=1 << 27), UNS), (dict(T=1 << 28), UNS),
]


@pytest.mark.parametrize("kw,code", DIMS)
def test_dims(L, kw, code):
    assert _plan(L, _dims(**kw)) == code
    assert _write(L, _dims(**kw)) == code


@pytest.mark.parametrize("kw", [
    dict(new=None), dict(off=None), dict(pos=None), dict(slots=None), dict(kv_len=None), dict(first=None),
    dict(pages=None), dict(free_pages=None), dict(n_free=None), dict(new=ODD), dict(off=ODD), dict(pos=ODD),
    dict(slots=ODD), dict(kv_len=ODD), dict(pages=ODD),
])
def test_plan_pointers(L, kw):
    assert _plan(L, **kw) == INV


def test_plan_needs_what_it_uses(L):
    assert _plan(L, _dims(T=0), pos=None, slots=None, off=None) == INV
    assert _plan(L, _dims(B=0), n_free=None) == INV
    assert L.moe_kv_plan(OK, ctypes.byref(_dims()), None, OK, OK, OK, 1 << 20, 256, None) == INV
    assert L.moe_kv_plan(OK, None, None, OK, OK, OK, 1 << 20, 256, None) == INV


@pytest.mark.parametrize("ws,n", [(None, 256), (1 << 20, 255), ((1 << 20) + 16, 256)])
def test_workspaces(L, ws, n):
    assert _plan(L, ws=ws, n=n) == WS
    assert _rows(L, ws=ws, n=n) == WS
    assert _write(L, ws=ws, n=n) == WS
    need = moe.moe_linear_fp4_workspace_bytes(4, 256, 128)
    assert _linear(L, ws=ws, n=need if n == 256 and ws else n) == WS
    assert _linear(L, n=need - 1) == WS


CONFIG = dict(base=10000.0, factor=4.0, orig_len=2048.0, lo=1.0, hi=32.0, magnitude=1.0, rot=64, scaling=0)


@pytest.mark.parametrize("kw,code", [
    (dict(base=1.0), INV), (dict(base=math.nan), INV), (dict(base=math.inf), INV), (dict(magnitude=0.0), INV),
    (dict(magnitude=-1.0), INV), (dict(magnitude=math.nan), INV), (dict(magnitude=1e39), INV), (dict(rot=0), INV), (dict(rot=-16), INV),
    (dict(scaling=4), INV), (dict(scaling=-1), INV), (dict(scaling=1, factor=0.5), INV),
    (dict(scaling=1, factor=math.nan), INV), (dict(scaling=2, orig_len=0.0), INV), (dict(scaling=2, lo=0.0), INV),
    (dict(scaling=2, lo=32.0), INV), (dict(scaling=3, hi=math.inf), INV), (dict(scaling=3, lo=math.nan), INV),
    (dict(rot=24), UNS), (dict(rot=272), UNS),
])
def test_rope_config(L, kw, code):
    g = moe.RopeConfig(**{**CONFIG, **kw})
    assert L.moe_rope_table(ctypes.byref(g), 0, 10, OK, None) == code


@pytest.mark.parametrize("pos0,n,table,code", [
    (-1, 10, OK, INV), (0, -1, OK, INV), (2**31 - 1, 2, OK, INV), (0, 10, None, INV), (0, 10, BAD, INV), (0, 0, None, OK_),
])
def test_rope_table(L, pos0, n, table, code):
    assert L.moe_rope_table(ctypes.byref(moe.RopeConfig(**CONFIG)), pos0, n, table, None) == code


def test_rope_table_null(L):
    assert L.moe_rope_table(None, 0, 10, OK, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(table=None), INV), (dict(table=BAD), INV), (dict(q_norm=BAD), INV), (dict(k_norm=BAD), INV),
    (dict(n_pos=-1), INV), (dict(rot=0), INV), (dict(rot=144), INV), (dict(flags=4), INV), (dict(eps=-1.0), INV),
    (dict(eps=math.nan), INV), (dict(rot=40), UNS),
])
def test_rope(L, kw, code):
    assert _rows(L, _rope(**kw)) == code
    assert _write(L, r=_rope(**kw)) == code


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), INV), (dict(x=BAD), INV), (dict(out=None), INV), (dict(out=BAD), INV), (dict(pos=None), INV),
    (dict(pos=ODD), INV), (dict(ldx=1016), INV), (dict(ldx=1028), INV), (dict(ldo=1016), INV),
    (dict(out=OK, ldo=1032), INV), (dict(T=-1), INV), (dict(H=0), INV), (dict(D=0), INV), (dict(D=96), UNS),
    (dict(D=256), UNS), (dict(T=1 << 28), UNS), (dict(T=0, x=None, pos=None, out=None), OK_),
])
def test_rope_rows(L, kw, code):
    assert _rows(L, **kw) == code


def test_rope_null(L):
    assert L.moe_rope_rows(OK, 1024, OK, 4, 8, 128, None, OK, 1024, 1 << 20, 256, None) == INV
    assert L.moe_rope_kv_write(OK, 1024, OK, 256, OK, 256, OK, OK, None, ctypes.byref(_dims()), ctypes.byref(_cache()),
                               OK, 1024, 1 << 20, 256, None) == INV


@pytest.mark.parametrize("kw,code", [
    (dict(q=None), INV), (dict(k=None), INV), (dict(v=None), INV), (dict(out=None), INV), (dict(q=BAD), INV),
    (dict(k=BAD), INV), (dict(v=BAD), INV), (dict(out=BAD), INV), (dict(pos=None), INV), (dict(slots=None), INV),
    (dict(pos=ODD), INV), (dict(slots=ODD), INV), (dict(ldq=1016), INV), (dict(ldk=248), INV), (dict(ldv=260), INV),
    (dict(ldo=1000), INV), (dict(out=OK, ldo=1032), INV), (dict(c=_cache(k=None)), INV), (dict(c=_cache(ks=None)), INV),
    (dict(c=_cache(slot_stride=136)), INV), (dict(d=_dims(T=0), q=None, pos=None, slots=None), OK_),
])
def test_rope_kv_write(L, kw, code):
    assert _write(L, **kw) == code


def _norm(L, dims=None, y=OK, res=OK, gate=None, w_post=OK, w_pre=OK, out=OK, x=OK, **kw):
    base = dict(T=4, d=256, gate=0, flags=0, eps=1e-6, scale=1.0)
    base.update(kw)
    return L.moe_block_norm(y, res, gate, w_post, w_pre, ctypes.byref(dims or moe.NormDims(**base)), out, x, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(d=0), INV), (dict(gate=4), INV), (dict(gate=-1), INV), (dict(flags=4), INV), (dict(eps=-1.0), INV),
    (dict(eps=math.inf), INV), (dict(scale=math.nan), INV), (dict(scale=math.inf), INV),
])
def test_norm_numbers(L, kw, code):
    kw = dict(kw)
    if "gate" in kw:
        d = moe.NormDims(T=4, d=256, gate=kw["gate"], flags=0, eps=0, scale=1)
        assert _norm(L, d, gate=OK) == code
    else:
        assert _norm(L, **kw) == code


@pytest.mark.parametrize("d", [4, 12, 32776])
def test_norm_widths(L, d):
    assert _norm(L, moe.NormDims(T=4, d=d, gate=0, flags=0, eps=0, scale=1)) == UNS


@pytest.mark.parametrize("kw", [
    dict(res=None), dict(res=BAD), dict(y=BAD), dict(w_post=BAD), dict(w_pre=BAD), dict(out=None), dict(out=BAD), dict(x=BAD),
    dict(x=None), dict(w_pre=None), dict(y=None), dict(y=None, w_post=None, w_pre=None, x=None), dict(gate=OK),
])
def test_norm_pointers(L, kw):
    assert _norm(L, **kw) == INV


@pytest.mark.parametrize("kind,ptr", [(1, None), (1, ODD), (2, BAD), (3, BAD), (3, None)])
def test_norm_gates(L, kind, ptr):
    d = moe.NormDims(T=4, d=256, gate=kind, flags=0, eps=0, scale=1)
    assert _norm(L, d, gate=ptr) == INV
    assert _norm(L, d, gate=OK, y=None, w_post=None) == INV


def test_norm_nothing_to_do(L):
    assert _norm(L, T=0) == OK_
    assert L.moe_block_norm(OK, OK, None, None, None, None, OK, None, None) == INV


def _linear(L, x=OK, ldx=128, T=4, N=256, K=128, q=OK, b=OK, s=OK, out=OK, ws=1 << 20, n=1 << 30):
    return L.moe_linear_fp4(x, ldx, T, N, K, moe.Fp4(q, b, s), out, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(N=0), INV), (dict(K=0), INV), (dict(K=-64), INV), (dict(K=96), UNS), (dict(K=65600), UNS),
    (dict(N=252), UNS), (dict(N=1 << 24), UNS), (dict(T=1 << 24), UNS), (dict(T=1 << 20, N=1 << 20), UNS), (dict(x=None), INV), (dict(x=BAD), INV),
    (dict(ldx=120), INV), (dict(ldx=132), INV), (dict(q=None), INV), (dict(q=BAD), INV), (dict(b=BAD), INV),
    (dict(s=ODD), INV), (dict(s=None), INV), (dict(out=None), INV), (dict(out=BAD), INV), (dict(T=0, x=None, out=None), OK_),
])
def test_linear(L, kw, code):
    assert _linear(L, **kw) == code


def test_fp4_sizes(L):
    assert moe.moe_fp4_scale_bytes(1, 64) == 512
    assert moe.moe_fp4_scale_bytes(129, 192) == 2 * 3 * 512
    assert moe.moe_fp4_scale_bytes(0, 64) == 0
    for rows, K in ((-1, 64), (1, 0), (1, 32), (1, 65600), (2**31 - 128, 64), (2**30, 65536)):
        assert moe.moe_fp4_scale_bytes(rows, K) == 0
    assert moe.moe_linear_fp4_workspace_bytes(1, 8, 64) > 256
    assert moe.moe_linear_fp4_workspace_bytes(1, 9, 64) == 0
    assert moe.moe_linear_fp4_workspace_bytes(-1, 8, 64) == 0


@pytest.mark.parametrize("kw,code", [
    (dict(rows=-1), INV), (dict(K=0), INV), (dict(K=48), UNS), (dict(rows=2**31 - 128), UNS), (dict(src=None), INV),
    (dict(src=BAD), INV), (dict(q=None), INV), (dict(q=BAD), INV), (dict(b=None), INV), (dict(b=BAD), INV), (dict(s=None), INV), (dict(s=ODD), INV),
    (dict(rows=0, src=None), OK_), (dict(rows=2**24, K=65536), UNS),
])
def test_fp4_rows(L, kw, code):
    a = dict(src=OK, rows=4, K=128, q=OK, b=OK, s=OK)
    a.update(kw)
    args = (a["src"], a["rows"], a["K"], a["q"], a["b"], a["s"], None)
    assert L.moe_pack_fp4(*args) == code
    assert L.moe_quant_rows_fp4(*args) == code
    assert L.moe_unpack_fp4(moe.Fp4(a["q"], a["b"], a["s"]), a["rows"], a["K"], a["src"], None) == code


def test_the_binding_refuses_host_tensors():
    i = torch.zeros(2, dtype=torch.int32)
    f = torch.zeros(4, 16)
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        moe.kv_pages(i, i, torch.zeros(2, 3, dtype=torch.int32), i, i[:1])
    with pytest.raises((ValueError, RuntimeError, AssertionError)):
        moe.rope(f)
    with pytest.raises(ValueError):
        moe.rope(f[0])
    with pytest.raises(ValueError):
        moe.kv_pages(i, i, i, i, i)
    with pytest.raises(ValueError):
        moe.moe_rope_table(moe.RopeConfig(**CONFIG), 0, f)
    with pytest.raises(ValueError):
        moe.fp4(torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(5, dtype=torch.uint8), torch.zeros(4))
