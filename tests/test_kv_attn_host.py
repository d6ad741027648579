"""Refusals of the paged cache's calls and of its attention: every bad argument comes back as
its documented status (or a ValueError of the binding) before anything is enqueued."""
import ctypes

import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

INV, UNS, WS = moe.MOE_ERR_INVALID_ARG, moe.MOE_ERR_UNSUPPORTED, moe.MOE_ERR_WORKSPACE
OK, BAD = 1 << 21, (1 << 21) + 8     # addresses, never dereferenced


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


def _cache(**kw):
    base = dict(k=OK, v=OK, ks=OK, vs=OK, page_stride=4096, head_stride=2048, slot_stride=128)
    base.update(kw)
    return moe.Kv(**base)


def _write(L, d=None, c=None, k=OK, ldk=256, v=OK, ldv=256, slots=OK, ws=1 << 20, n=256):
    return L.moe_kv_write(k, ldk, v, ldv, slots, ctypes.byref(d or _dims()),
                          ctypes.byref(c or _cache()), ws, n, None)


def _read(L, d=None, c=None, slots=OK, k=OK, v=OK, ws=1 << 20, n=256):
    return L.moe_kv_read(slots, ctypes.byref(d or _dims()), ctypes.byref(c or _cache()), k, v, ws, n,
                         None)


def _attn(L, d=None, c=None, q=OK, ldq=1024, off=OK, lens=OK, pages=OK, scale=0.1, out=OK, lse=None,
          ws=1 << 20, n=None):
    d = d or _dims()
    n = moe.moe_attn_workspace_bytes(d) if n is None else n
    return L.moe_attn_paged(q, ldq, off, lens, pages, ctypes.byref(d), ctypes.byref(c or _cache()),
                            scale, out, lse, ws, n, None)


@pytest.mark.parametrize("kw,code", [
    (dict(T=-1), INV), (dict(B=-1), INV), (dict(H=0), INV), (dict(H_kv=0), INV), (dict(H=7), INV),
    (dict(page=0), INV), (dict(n_pages=0), INV), (dict(max_pages=0), INV), (dict(max_new=-1), INV),
    (dict(window=-1), INV), (dict(D=0), INV),
    (dict(D=96), UNS), (dict(D=256), UNS), (dict(page=8), UNS), (dict(page=48), UNS),
    (dict(page=512), UNS), (dict(format=3), UNS), (dict(format=-1), UNS), (dict(H=258, H_kv=2), UNS),
    (dict(B=8193), UNS), (dict(n_pages=1 << 27), UNS), (dict(max_pages=1 << 27), UNS),
    (dict(T=1 << 28), UNS),
])
def test_dims(L, kw, code):
    d = _dims(**kw)
    assert moe.moe_attn_workspace_bytes(d) == 0
    big = 1 << 30
    assert _write(L, d, n=big) == code
    assert _read(L, d, n=big) == code
    assert _attn(L, d, n=big) == code


def test_null_dims(L):
    assert L.moe_kv_write(OK, 256, OK, 256, OK, None, None, OK, 256, None) == INV
    assert L.moe_kv_read(OK, None, None, OK, OK, OK, 256, None) == INV
    assert L.moe_attn_paged(OK, 1024, OK, OK, OK, None, None, 1.0, OK, None, OK, 1 << 30, None) == INV


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=BAD), dict(v=BAD), dict(ks=None), dict(vs=None),
    dict(ks=OK + 2), dict(vs=OK + 2), dict(page_stride=0), dict(head_stride=-2048),
    dict(slot_stride=136), dict(page_stride=1 << 40),
])
def test_cache(L, kw):
    c = _cache(**kw)
    assert _write(L, c=c) == INV
    assert _read(L, c=c) == INV
    assert _attn(L, c=c) == INV


def test_write_and_read_arguments(L):
    for kw in (dict(k=None), dict(k=BAD), dict(v=BAD), dict(ldk=255), dict(ldk=248), dict(ldv=260),
               dict(slots=None)):
        assert _write(L, **kw) == INV, kw
    for kw in (dict(k=None), dict(v=BAD), dict(slots=None)):
        assert _read(L, **kw) == INV, kw
    for call in (_write, _read):
        assert call(L, ws=None) == WS
        assert call(L, ws=(1 << 20) + 16) == WS
        assert call(L, n=255) == WS


def test_attention_arguments(L):
    for kw in (dict(q=None), dict(q=BAD), dict(ldq=1020), dict(ldq=1016), dict(off=None),
               dict(lens=None), dict(pages=None), dict(out=None), dict(out=BAD), dict(lse=OK + 2),
               dict(scale=float("nan")), dict(scale=float("inf")), dict(d=_dims(B=0))):
        assert _attn(L, **kw) == INV, kw
    assert _attn(L, ws=None) == WS
    assert _attn(L, ws=(1 << 20) + 16) == WS
    assert _attn(L, n=moe.moe_attn_workspace_bytes(_dims()) - 1) == WS


def test_no_tokens_is_ok(L):
    d = _dims(T=0)
    assert _write(L, d, k=None, v=None, slots=None) == moe.MOE_OK
    assert _read(L, d, k=None, v=None, slots=None) == moe.MOE_OK
    assert _attn(L, d, q=None, out=None) == moe.MOE_OK
    assert _attn(L, _dims(T=0, D=96), n=1 << 30) == UNS


def test_binding_checks_shapes(L):
    z = torch.zeros
    with pytest.raises(ValueError):
        moe.kv_cache(z(2, 2, 16, 128, dtype=torch.bfloat16), z(2, 2, 16, 128, dtype=torch.bfloat16))
    d, c = _dims(), _cache()
    with pytest.raises(ValueError):
        moe.moe_kv_write(z(4, 2, 128), z(4, 2, 128), z(4, dtype=torch.int32), d, c, z(256))
    with pytest.raises(ValueError):
        moe.moe_attn_paged(z(4, 8, 128), z(3), z(2), z(2, 4), d, c, 1.0, z(4, 8, 128), None, z(256))
