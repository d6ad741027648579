"""Tokens planned and dropped again where a window gives pages back meanwhile: what is as before, and what is not."""
import random

import pytest
import torch

from test_gpu_kv_plan import Device, Pool, both

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("window,page", [(1, 16), (20, 16), (30, 32)])
@pytest.mark.parametrize("seed", range(3))
def test_added_and_dropped_with_a_window(window, page, seed):
    rng = random.Random(seed)
    B = 9
    dev = Device(Pool(B, page, 200, 20, window, seed))
    for _ in range(3):
        both(dev, [rng.randrange(0, 40) for _ in range(B)], 400, tripped=False)
    kv_len, first, pages = (t.clone() for t in (dev.kv_len, dev.first, dev.pages))
    new = [rng.randrange(0, 60) for _ in range(B)]
    both(dev, new, 600, tripped=False)
    gave = int((dev.first - first).sum())
    first_then = dev.first.clone()
    dropped = [-n if n else 0 for n in new]
    both(dev, dropped, 0)
    # lengths are those of before; so are the entries of all pages but those that the window gave back, which stay free
    kept = dev.kv_len == kv_len
    assert all(kept.tolist())
    assert torch.equal(dev.first, first_then)
    for b in range(B):
        want = pages[b].clone()
        want[: first_then[b]] = -1
        if kv_len[b] == 0:
            want[:] = -1
        assert torch.equal(dev.pages[b], want)
    assert gave > 0
    # and the next step finds them
    both(dev, new, 600, tripped=False)
