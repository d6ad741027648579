"""The norms between blocks where a CTA or warp walks many rows: every row bit for bit what a call gives that has a row for each
CTA, and rows of either end of the walks against the formulas in 64 bits."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from test_gpu_block_norm import EPS, check, inputs

pytestmark = pytest.mark.gpu


def call(args, dims, r_out, x):
    y, res, gate, w_post, w_pre = args
    moe.moe_block_norm(y, res, gate, w_post, w_pre, dims, r_out, x)


def outputs(args):
    y, res, _, _, w_pre = args
    return (None if y is None else torch.full_like(res, 7.0),
            None if w_pre is None else torch.full(res.shape, 7.0, dtype=torch.bfloat16, device="cuda"))


def rows_of(args, dims, rows):
    """The same call on some of the rows."""
    y, res, gate, w_post, w_pre = args
    take = lambda t: None if t is None else t[rows].contiguous()  # noqa: E731
    return ((take(y), take(res), take(gate) if dims.gate in (moe.MOE_GATE_TOKEN, moe.MOE_GATE_FULL) else gate, w_post, w_pre),
            moe.NormDims(T=len(range(dims.T)[rows]) if isinstance(rows, slice) else len(rows), d=dims.d, gate=dims.gate,
                         flags=dims.flags, eps=dims.eps, scale=dims.scale))


def equal(a, b):
    return a is None and b is None or torch.equal(a.view(torch.uint8), b.view(torch.uint8))


# Rows of a warp with 16 and 32 elements to a lane, of a CTA with up to 640 and with 1024 threads; `per`: rows that an SM
# has at work at once at most, so that every warp or CTA takes three or more (and one or three of them are on the way).
SHAPES = [(264, 32), (1000, 32), (2048, 4), (4096, 4), (6000, 4), (9000, 1), (16384, 1)]


# norms after and before, and the first norm of a model, which has no gate
PARTS = [(kind, res32, post, pre, False) for kind, res32 in ((0, False), (1, True), (2, False), (3, False), (3, True))
         for post in (True, False) for pre in (True, False)] + [(0, False, False, True, True), (0, True, False, True, True)]


@pytest.mark.parametrize("kind,res32,post,pre,first", PARTS)
@pytest.mark.parametrize("d,per", SHAPES)
def test_walks(d, per, kind, res32, post, pre, first):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    T = 5 * per * sms + 7
    flags = (moe.MOE_NORM_RESIDUAL_F32 if res32 else 0) | (moe.MOE_NORM_SIGMOID if kind == 2 else 0)
    dims = moe.NormDims(T=T, d=d, gate=kind, flags=flags, eps=EPS, scale=0.7)
    base = inputs(64, d, kind, post, pre, res32, seed=d + kind, y=not first)
    # many rows out of few, none like another: signs and sizes by position
    g = torch.Generator(device="cuda").manual_seed(d)
    pick = torch.randint(0, 64, (T,), generator=g, device="cuda")
    size = torch.exp2(torch.randint(-3, 4, (T, 1), generator=g, device="cuda").float())
    spread = lambda t: None if t is None else (t[pick].float() * size).to(t.dtype)  # noqa: E731
    y, res, gate, w_post, w_pre = base
    gate = gate if kind in (0, 2) else (gate[pick] * size.view(-1) if kind == 1 else spread(gate))
    args = (spread(y), spread(res), gate, w_post, w_pre)
    r, x = outputs(args)
    call(args, dims, r, x)
    for lo in range(0, T, sms):
        some, few = rows_of(args, dims, slice(lo, min(lo + sms, T)))
        r1, x1 = outputs(some)
        call(some, few, r1, x1)
        assert equal(r1, None if r is None else r[lo:lo + sms]) and equal(x1, None if x is None else x[lo:lo + sms])
    ends = list(range(40)) + list(range(T - 40, T))
    some, few = rows_of(args, dims, ends)
    check(*some, few, None if r is None else r[ends], None if x is None else x[ends])
    # in place: the rows to come are on the way while a row's outputs take its inputs' place
    keep = [None if t is None else t.clone() for t in args]
    call(args, dims, None if first else args[1], None if x is None else args[0] if not first else x)
    assert first or equal(args[1], r)
    if x is not None and not first:
        assert equal(args[0], x)
    if first:
        assert equal(args[1], keep[1])
