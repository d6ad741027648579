"""A whole decode step, as the example composes it: every call held to its definition, and captured steps equal to
plain ones."""
import math
import os
import sys

import pytest
import torch

import attn_cases as ac
import test_gpu_block_norm as norms
import test_gpu_fp4 as fp4
import test_gpu_rope as ropes

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt", ac.FORMATS)
def test_captured_steps(fmt):
    import decode_step
    off, same, lengths = decode_step.main(fmt)
    # 91 steps: prompts and a token each; the second begins anew, the third drops three tokens at one step instead of adding one
    assert off == 0.0 and same and lengths == [19 + 90, 23 + 58, 14 + 89 - 3]


def _unpacked(w, rows):
    """What packed weights stand for, in 64 bits, on the CPU."""
    q, tiles, s = (t.cpu() for t in w.tensors)
    K = 2 * q.shape[1]
    codes = torch.stack((q & 15, q >> 4), -1).view(rows, K).long()
    b = tiles.view(-1, K // 64, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(-1, K // 16)[:rows].long()
    return fp4.values(codes, b, s)[0], s.double()


def _projected(x, w, out):
    """A projection held to the sums of what its codes stand for."""
    N, K = w.shape
    c, b, sx = fp4.recipe(x)
    xv, (wv, sw) = fp4.values(c, b, sx)[0], _unpacked(w, N)
    scale = sx.double()[:, None] * sw
    want, size = xv @ wv.T * scale, xv.abs() @ wv.abs().T * scale
    assert ((out.cpu().double() - want).abs() <= 2.0 ** -8 * want.abs() + (K + 8) * 2.0 ** -23 * size + 1e-37).all()


@pytest.mark.parametrize("fmt", ac.FORMATS)
def test_each_call_of_a_step(fmt, monkeypatch):
    import decode_step as ex
    moe = ex.moe
    block = ex.Block(fmt, 3, 40)
    call = {n: getattr(moe, n) for n in ("moe_block_norm", "moe_linear_fp4", "moe_rope_kv_write", "moe_attn_paged")}
    seen = []

    def norm(y, residual, gate, w_post, w_pre, dims, residual_out, x):
        keep = [None if t is None else t.clone() for t in (y, residual, gate, w_post, w_pre)]
        call["moe_block_norm"](y, residual, gate, w_post, w_pre, dims, residual_out, x)
        norms.check(*keep, dims, residual_out, x)
        seen.append("norm")

    def linear(x, w, out, ws):
        call["moe_linear_fp4"](x, w, out, ws)
        _projected(x, w, out)
        seen.append("linear")

    def rope(q, k, v, pos, slots, rope, dims, cache, q_out, ws):
        was = [None if t is None else t.clone() for t in block.pool]
        before = q_out.clone()
        call["moe_rope_kv_write"](q, k, v, pos, slots, rope, dims, cache, q_out, ws)
        live = pos >= 0
        table, qn, kn = (t.cpu() for t in rope.tensors)
        row = table[pos[live].cpu().long()]
        room = 2.0 ** -17 * 2 * math.sqrt(ex.D)
        ropes.bf16_close(q_out[live], ropes.rotated(q[live].cpu(), qn, ex.EPS, row, rope.rot, False, dtype=torch.float64),
                         room * qn.abs().max().item())
        assert torch.equal(q_out[~live], before[~live])
        # values: the recipe bit for bit; keys within half a step of their code; no other slot changes
        p, at = slots[live].long() // ex.page, slots[live].long() % ex.page
        codes, s = ac.quantise(v[live], fmt)
        was[1][p, :, at] = codes
        if s is not None:
            was[3][p, :, at] = s
            assert torch.equal(block.pool[3], was[3])
        assert torch.equal(block.pool[1], was[1])
        want = ropes.rotated(k[live].cpu(), kn, ex.EPS, row, rope.rot, False, dtype=torch.float64)
        got = ac.values(block.pool[0][p, :, at], None if s is None else block.pool[2][p, :, at], fmt).double().cpu()
        top = want.abs().amax(-1, keepdim=True)
        step = {"bf16": want.abs() * 2.0 ** -8, "e4m3": torch.maximum(want.abs() * 2.0 ** -4, top / 448 * 2.0 ** -10),
                "int4": top / 14}[fmt]
        assert ((got - want).abs() <= step * (1 + 2.0 ** -8) + 2 * room * kn.abs().max().item()).all()
        was[0][p, :, at] = block.pool[0][p, :, at]
        assert torch.equal(block.pool[0], was[0])
        seen.append("rope")

    def attn(q, q_off, kv_len, pages, dims, cache, scale, out, lse, ws):
        T = q_off[-1].item()
        z = torch.full((dims.T, dims.H), 7.0, device="cuda")
        call["moe_attn_paged"](q, q_off, kv_len, pages, dims, cache, scale, out, z, ws)
        k, v, ks, vs = block.pool
        ac.check(ac.Batch(q_off.diff().tolist(), kv_len.tolist(), dims.H, dims.H_kv, dims.D, dims.page, fmt, dims.window,
                          scale, q[:T], q_off, kv_len, pages, k, v, ks, vs), out[:T], z[:T])
        seen.append("attn")

    for name, f in (("moe_block_norm", norm), ("moe_linear_fp4", linear), ("moe_rope_kv_write", rope), ("moe_attn_paged", attn)):
        monkeypatch.setattr(moe, name, f)
    g = torch.Generator(device="cuda").manual_seed(9)
    for new in ([19, 0, 14], [1, 20, 1], [1, 1, -4], [-(1 << 31), 1, 30], [25, 1, 1]):
        block.new.copy_(torch.tensor(new, dtype=torch.int32))
        block.residual.copy_(torch.randn((40, ex.d), generator=g, device="cuda").to(torch.bfloat16))
        block.step()
        assert block.status() == [moe.MOE_OK] * 3
    assert seen == ["norm", "linear", "rope", "attn", "linear", "norm", "norm"] * 5
    assert block.kv_len.tolist() == [25, 23, 14 + 1 - 4 + 30 + 1]
