"""Plans of as many rows as there can be: what names them is sized in 64 bits."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [2**31 - 1, 2**31 - 4])
def test_most_rows(T):
    ints = lambda v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    kv_len, first, free, n_free = ints([15, 0]), ints([0, 0]), ints([5, 4, 3, 2, 1, 6]), ints([5])
    pages = ints([[0, -1, -1], [-1, -1, -1]])
    st, ws = moe.kv_pages(kv_len, first, pages, free, n_free), moe.workspace(256)
    dims = moe.KvDims(T=T, B=2, H=1, H_kv=1, D=64, page=16, n_pages=6, max_pages=3, max_new=0, window=0, format=0, flags=0)
    q_off, pos, slots = ints([7] * 3), *(torch.zeros(T, dtype=torch.int32, device="cuda") for _ in range(2))
    moe.moe_kv_plan(ints([3, 2]), dims, st, q_off, pos, slots, ws)
    assert moe.moe_check_device_status(ws) == moe.MOE_OK
    assert q_off.tolist() == [0, 3, 5] and kv_len.tolist() == [18, 2]
    assert pos[:5].tolist() == [15, 16, 17, 0, 1] and slots[:5].tolist() == [15, 16, 17, 32, 33]
    assert pages.tolist() == [[0, 1, -1], [2, -1, -1]] and n_free.tolist() == [3]
    for t in (pos, slots):
        for lo in range(5, T, 1 << 28):
            assert (t[lo:lo + (1 << 28)] == -1).all()
