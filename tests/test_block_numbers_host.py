"""Numbers that do not fit the C ABI's 32 bits are refused by the binding, not cut."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_sigmoid_gb300.build as b
    b.build()


class Table:
    """What the binding asks of a table on device 0; no memory behind it."""
    shape, dtype = torch.Size((4, 64)), torch.float32

    def get_device(self):
        return 0

    def numel(self):
        return 256

    def dim(self):
        return 2

    def is_contiguous(self):
        return True

    def data_ptr(self):
        return 1 << 21


@pytest.mark.parametrize("pos0", [1 << 31, (1 << 32) + 5, -(1 << 32)])
def test_first_positions(pos0, monkeypatch):
    monkeypatch.setattr(moe, "_current_device", lambda: 0)
    called = []
    monkeypatch.setattr(moe, "_lib", type("L", (), {"moe_rope_table": staticmethod(lambda *a: called.append(a) or 0)}))
    g = moe.RopeConfig(base=10000.0, factor=1.0, orig_len=1.0, lo=1.0, hi=2.0, magnitude=1.0, rot=64, scaling=0)
    stream = type("S", (), {"cuda_stream": 0})
    with pytest.raises(ValueError):
        moe.moe_rope_table(g, pos0, Table(), stream=stream)
    assert not called
    moe.moe_rope_table(g, (1 << 31) - 4, Table(), stream=stream)
    assert called[0][1] == (1 << 31) - 4


@pytest.mark.parametrize("sizes", [((1 << 32) + 1, 8, 64), (1, (1 << 32) + 8, 64), (1, 8, (1 << 32) + 64), (1 << 31, 8, 64)])
def test_workspaces_of_refused_sizes(sizes):
    assert moe.moe_linear_fp4_workspace_bytes(*sizes) == 0


@pytest.mark.parametrize("sizes", [((1 << 64) + 1, 64), (1, (1 << 64) + 64)])
def test_scales_of_refused_sizes(sizes):
    assert moe.moe_fp4_scale_bytes(*sizes) == 0
