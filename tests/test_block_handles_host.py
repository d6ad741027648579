"""Handles of another device's tensors, and workspaces that are not one run of bytes, are refused before anything is enqueued.
Stand-ins for CUDA tensors: nothing here has memory on a device."""
import types

import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

STREAM = types.SimpleNamespace(cuda_stream=0)


class Stand:
    """What the binding asks of a tensor."""
    is_cuda = True

    def __init__(self, shape, dtype, dev=0, contiguous=True):
        self.shape, self.dtype, self.dev, self.contiguous = torch.Size(shape), dtype, dev, contiguous

    def get_device(self):
        return self.dev

    def numel(self):
        return self.shape.numel()

    def dim(self):
        return len(self.shape)

    def element_size(self):
        return torch.empty((), dtype=self.dtype).element_size()

    @property
    def nbytes(self):
        return self.numel() * self.element_size()

    def is_contiguous(self):
        return self.contiguous

    def stride(self, i=None):
        s, n = [], 1
        for v in reversed(self.shape):
            s.insert(0, n)
            n *= v
        return tuple(s) if i is None else s[i]

    def data_ptr(self):
        return 1 << 21


@pytest.fixture(scope="module", autouse=True)
def built():
    import moe_expert_layer_sigmoid_gb300.build as b
    b.build()


@pytest.fixture
def on(monkeypatch):
    """Makes a device the current one."""
    def go(dev):
        monkeypatch.setattr(moe, "_current_device", lambda: dev)
    go(0)
    return go


I, F, U, H = torch.int32, torch.float32, torch.uint8, torch.bfloat16
T, HEADS, H_KV, D, B, PAGE, N_PAGES, MAX_PAGES = 4, 4, 2, 64, 3, 16, 10, 5
DIMS = moe.KvDims(T=T, B=B, H=HEADS, H_kv=H_KV, D=D, page=PAGE, n_pages=N_PAGES, max_pages=MAX_PAGES, max_new=0, window=0,
                  format=moe.MOE_KV_E4M3, flags=0)


def handles(dev):
    return types.SimpleNamespace(
        pages=moe.kv_pages(Stand((B,), I, dev), Stand((B,), I, dev), Stand((B, MAX_PAGES), I, dev), Stand((N_PAGES,), I, dev),
                           Stand((1,), I, dev)),
        rope=moe.rope(Stand((100, 32), F, dev)),
        w=moe.fp4(Stand((64, 64), U, dev), Stand((moe.moe_fp4_scale_bytes(64, 128),), U, dev), Stand((64,), F, dev)),
        cache=moe.kv_cache(Stand((N_PAGES, H_KV, PAGE, D), U, dev), Stand((N_PAGES, H_KV, PAGE, D), U, dev),
                           Stand((N_PAGES, H_KV, PAGE), F, dev), Stand((N_PAGES, H_KV, PAGE), F, dev)))


def calls(h, ws):
    q, kv = Stand((T, HEADS, D), H), Stand((T, H_KV, D), H)
    return dict(
        pages=lambda: moe.moe_kv_plan(Stand((B,), I), DIMS, h.pages, Stand((B + 1,), I), Stand((T,), I), Stand((T,), I), ws,
                                      stream=STREAM),
        rope=lambda: moe.moe_rope_rows(q, Stand((T,), I), h.rope, Stand((T, HEADS, D), H), ws, stream=STREAM),
        write=lambda: moe.moe_rope_kv_write(q, kv, kv, Stand((T,), I), Stand((T,), I), h.rope, DIMS, h.cache,
                                            Stand((T, HEADS, D), H), ws, stream=STREAM),
        w=lambda: moe.moe_linear_fp4(Stand((T, 128), H), h.w, Stand((T, 64), H), ws, stream=STREAM))


@pytest.mark.parametrize("handle,call", [("pages", "pages"), ("rope", "rope"), ("rope", "write"), ("cache", "write"), ("w", "w")])
def test_handles_of_another_device(on, handle, call):
    ours = handles(0)
    on(1)
    theirs = handles(1)
    on(0)
    setattr(ours, handle, getattr(theirs, handle))
    with pytest.raises(ValueError, match="device"):
        calls(ours, Stand((1 << 20,), U))[call]()


@pytest.mark.parametrize("call", ["pages", "rope", "write", "w"])
def test_workspaces(on, call):
    with pytest.raises(ValueError, match="ws"):
        calls(handles(0), Stand((1 << 20,), U, contiguous=False))[call]()
    with pytest.raises(ValueError, match="ws"):
        calls(handles(0), Stand((1 << 20,), U, dev=1))[call]()


def test_a_cache_of_two_devices(on):
    with pytest.raises(ValueError, match="device"):
        moe.kv_cache(Stand((2, 1, 16, 64), U), Stand((2, 1, 16, 64), U), Stand((2, 1, 16), F), Stand((2, 1, 16), F, dev=1))
