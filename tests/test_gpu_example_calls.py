"""Every call that the decoder block example makes of the cache and the attention, held to its definition:
rows as they are written bit for bit, outputs element by element against 64 bits over what the cache holds."""
import os
import sys

import pytest
import torch

import attn_cases as ac

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("seed", [0, 1])
def test_each_call_of_the_example(fmt, seed, monkeypatch):
    import decoder_block as ex
    moe, pools, rows, calls = ex.moe, {}, {}, []
    kv_cache, write, attn = moe.kv_cache, moe.moe_kv_write, moe.moe_attn_paged

    def spy_cache(*tensors):
        c = kv_cache(*tensors)
        pools[id(c)] = (c, tensors)
        rows[id(c)] = {}
        return c

    def spy_write(k, v, slots, dims, cache, ws):
        tensors = pools[id(cache)][1]
        want = [None if t is None else t.clone() for t in tensors]
        write(k, v, slots, dims, cache, ws)
        p, at = slots.long() // dims.page, slots.long() % dims.page
        for x, pool, scales in ((k, 0, 2), (v, 1, 3)):
            codes, s = ac.quantise(x, fmt)
            want[pool][p, :, at] = codes
            if s is not None:
                want[scales][p, :, at] = s
        for t, w in zip(tensors, want):
            assert t is None or torch.equal(t, w)
        for i, s in enumerate(slots.tolist()):
            assert s not in rows[id(cache)], "a slot written twice"
            rows[id(cache)][s] = torch.stack((k[i], v[i])).clone()

    def spy_attn(q, q_off, kv_len, pages, dims, cache, scale, out, lse, ws):
        assert lse is None
        z = torch.full((dims.T, dims.H), 7.0, device="cuda")
        attn(q, q_off, kv_len, pages, dims, cache, scale, out, z, ws)
        new, total = q_off.diff().tolist(), kv_len.tolist()
        k, v, ks, vs = pools[id(cache)][1]
        ac.check(ac.Batch(new, total, dims.H, dims.H_kv, dims.D, dims.page, fmt, dims.window, scale, q, q_off, kv_len,
                          pages, k, v, ks, vs), out, z)
        # all the keys that the sequences have by now lie in the pages that the call was given
        held = {int(p) * dims.page + j % dims.page for b, t in enumerate(total) for j in range(t)
                for p in [pages[b, j // dims.page]]}
        assert held == set(rows[id(cache)]) and len(held) == sum(total)
        calls.append(sum(new))

    monkeypatch.setattr(moe, "kv_cache", spy_cache)
    monkeypatch.setattr(moe, "moe_kv_write", spy_write)
    monkeypatch.setattr(moe, "moe_attn_paged", spy_attn)
    ex.main(fmt, seed=seed)
    assert len(calls) > 10 and max(calls) == 116 and min(calls) == 1
    # Both blocks are given the same rows, whole and in chunks.  Their projections are products of 256 terms
    # summed in another order, each sum off by 256 * 2^-24 * sum |x w| at most, rounded to bf16 (2^-8 each);
    # sum |x w| is at most the norms' product: 16 for a normalised row, below 2 for a column of unit variance.
    a, b = rows.values()
    assert a.keys() == b.keys()
    for s in a:
        x, y = a[s].double(), b[s].double()
        assert ((x - y).abs() <= 2.0 ** -7 * torch.maximum(x.abs(), y.abs()) + 2 * 256 * 2.0 ** -24 * 32).all()
