"""A launch that CUDA refuses is told once, by the call that made it: the next call starts clean."""
import os
import subprocess
import sys

import pytest

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# While a capture of a blocking stream is open, CUDA refuses launches on the legacy stream.  (In a process of its own.)
PROGRAM = """
import ctypes, os, torch
import moe_expert_layer_sigmoid_gb300 as moe
home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
rt = ctypes.CDLL(next(p for p in (home + "/lib64/libcudart.so", home + "/targets/sbsa-linux/lib/libcudart.so") if os.path.exists(p)))
ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")
bf16 = lambda *s: torch.ones(s, dtype=torch.bfloat16, device="cuda")
st = moe.kv_pages(ints(0), ints(0), ints(-1, -1).view(1, 2), ints(0, 1), ints(2))
kv = moe.KvDims(T=1, B=1, H=1, H_kv=1, D=64, page=16, n_pages=2, max_pages=2, max_new=0, window=0, format=0, flags=0)
new, off, pos, slots, ws = ints(1), ints(0, 0), ints(0), ints(0), moe.workspace(256)
w = moe.fp4(*moe.moe_pack_fp4(torch.ones(64, 128, device="cuda")))
x4, out4, ws4 = bf16(8, 128), bf16(8, 64), moe.workspace(moe.moe_linear_fp4_workspace_bytes(8, 64, 128))
y, r, x = bf16(4, 256), bf16(4, 256), bf16(4, 256)
one, nd = torch.ones(256, device="cuda"), moe.NormDims(T=4, d=256, gate=0, flags=0, eps=1e-6, scale=1.0)
calls = dict(plan=lambda: moe.moe_kv_plan(new, kv, st, off, pos, slots, ws), linear=lambda: moe.moe_linear_fp4(x4, w, out4, ws4),
             norm=lambda: moe.moe_block_norm(y, r, None, one, one, nd, r, x))
for f in calls.values():
    f()
torch.cuda.synchronize()
s, graph = ctypes.c_void_p(), ctypes.c_void_p()
assert rt.cudaStreamCreate(ctypes.byref(s)) == 0
assert rt.cudaStreamBeginCapture(s, 0) == 0
try:
    calls["FIRST"]()
    raise SystemExit("the launch was not refused")
except moe.MoeError:
    pass
rt.cudaStreamEndCapture(s, ctypes.byref(graph))
rt.cudaGetLastError()
calls["NEXT"]()
torch.cuda.synchronize()
"""


@pytest.mark.parametrize("first", ["plan", "linear", "norm"])
@pytest.mark.parametrize("after", ["plan", "linear", "norm"])
def test_the_next_call(first, after):
    p = subprocess.run([sys.executable, "-c", PROGRAM.replace("FIRST", first).replace("NEXT", after)], cwd=ROOT,
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, p.stderr[-1500:]
