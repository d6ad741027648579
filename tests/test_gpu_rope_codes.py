"""Turned keys as codes where their scales are subnormal: the recipe bit for bit, its clamp included."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from attn_cases import quantise
from test_gpu_rope import _write_setup, config, rotated

pytestmark = pytest.mark.gpu


# A table's magnitude of 2^-149 times 7 to 3000: the largest of a row's turned elements is some units of 2^-149, and a
# scale of so few units is rounded by up to half of one, so that quotients pass the codes' largest value.
@pytest.mark.parametrize("fmt", ["int4", "e4m3"])
@pytest.mark.parametrize("units", [2, 7, 40, 700, 3000])
@pytest.mark.parametrize("pairs", [False, True])
def test_keys_of_subnormal_scales(units, fmt, pairs):
    T, H, H_kv, D, page = 64, 4, 2, 64, 16
    q, k, v, slots, pos, pool, sc, dims, cache = _write_setup(T, H, H_kv, D, page, fmt, "heads", seed=units)
    table, ws = torch.empty(2000, D, device="cuda"), moe.workspace(256)
    moe.moe_rope_table(config(rot=D, magnitude=units * 2.0 ** -149), 0, table)
    out = torch.empty(T, H, D, dtype=torch.bfloat16, device="cuda")
    moe.moe_rope_kv_write(q, k, v, pos.cuda(), slots.cuda(), moe.rope(table, moe.MOE_ROPE_PAIRS if pairs else 0), dims, cache,
                          out, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    turned = rotated(k.cpu(), None, 0, table.cpu()[pos.long()], D, pairs)
    codes, scales = quantise(turned, fmt)
    p, at = slots.long() // page, slots.long() % page
    assert torch.equal(sc[0].cpu()[p, :, at], scales)
    assert torch.equal(pool[0].cpu()[p, :, at], codes)
    if (units, fmt) in ((7, "int4"), (700, "e4m3")):      # (the cases reach past the largest code)
        top = turned.double().abs().amax(-1) / scales.double()
        assert (top[scales > 0] > {"int4": 7.5, "e4m3": 464}[fmt]).any()
