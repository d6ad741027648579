"""Attention over the paged cache at the edges of what a call may hold."""
import pytest
import torch

import attn_cases as ac
import moe_expert_layer_sigmoid_gb300 as moe
from test_gpu_attn_paged import ok, run

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("end", [-2 ** 31, -2 ** 31 + 4, -1, 2 ** 31 - 1])
@pytest.mark.parametrize("n", [4, 60])
def test_offsets_that_hold_anything(fmt, end, n):
    """Offsets whose difference does not fit 32 bits: the two sequences that share one are left out and
    recorded, the others are as ever."""
    b = ac.make([5, n, 3, 1, 40], [30, 70, 20, 50, 90], 8, 2, 64, 16, fmt, seed=3)
    b.q_off[2] = end
    out, lse, ws = run(b)
    assert moe.moe_check_device_status(ws) == moe.MOE_ERR_DEVICE_CHECK
    ref, z, bo, bl = ac.reference(b)
    at = torch.tensor(list(range(5)) + list(range(8 + n, 49 + n)), device="cuda")
    assert ((out.double() - ref)[at].abs() <= bo[at]).all()
    assert ((lse.double() - z)[at].abs() <= bl[at]).all()
    assert (out[5:8 + n] == 7).all() and (lse[5:8 + n] == 7).all()


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 4, 2 ** 30, 130, 3])
@pytest.mark.parametrize("G", [1, 4, 24])
def test_windows_with_tokens_before_the_start(fmt, window, G):
    """A window of any size, the largest standing for none, where some tokens sit before the start."""
    new = [10, 3, 1, 200, 40, 1]
    total = [5, 1, 0, 100, 17, 300]
    ok(ac.make(new, total, 2 * G, 2, 128, 16, fmt, window=window, seed=G))


@pytest.mark.parametrize("fmt", ac.FORMATS)
@pytest.mark.parametrize("new", [1, 3, 100, 250])
@pytest.mark.parametrize("page,left", [(64, 0), (64, 10), (16, 0), (16, 7)])
def test_the_longest_length(fmt, new, page, left):
    """Sequences that end within a tile of 2^31 keys, seen through a window; behind the last key of the page
    lies what must never matter."""
    far = 2 ** 31 - page          # keys of the longest page table
    total = far - left
    window, near = 300, 2048      # keys the window can reach, in whole pages
    b = ac.make([new], [near - left], 8, 2, 64, page, fmt, window=window, seed=new)
    # the same pages at the end of a page table of 2^31 keys: positions are 2^31 less a constant
    pages = torch.full((1, far // page), 0x7FFFFFF0, dtype=torch.int32, device="cuda")
    pages[0, -(near // page):] = b.pages[0, :near // page]
    ref = ac.reference(b)
    dims = b.dims(moe, max_pages=far // page)
    b.pages = pages
    b.kv_len.fill_(total)
    out, lse, ws = run(b, dims=dims)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    assert ((out.double() - ref[0]).abs() <= ref[2]).all()
    assert ((lse.double() - ref[1]).abs() <= ref[3]).all()
