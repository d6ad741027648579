"""The calls around the attention and the experts where no device answers: each comes back with MOE_ERR_CUDA and the process
lives on.  In a process of its own that sees no device; addresses are never dereferenced."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CALLS = {
    "moe_kv_plan": "[L.moe_kv_plan(A, i(d), i(st), A, A, A, W, 256, None)]",
    "moe_rope_table": "[L.moe_rope_table(i(g), 0, 10, A, None)]",
    "moe_rope_rows": "[L.moe_rope_rows(A, 1024, A, 4, 8, 128, i(r), A, 1024, W, 256, None)]",
    "moe_rope_kv_write": "[L.moe_rope_kv_write(A, 1024, A, 256, A, 256, A, A, i(r), i(d), i(c), A, 1024, W, 256, None)]",
    "moe_block_norm": "[L.moe_block_norm(A, A, None, A, A, i(moe.NormDims(T=4, d=n, gate=0, flags=0, eps=1e-6, scale=1.0)), "
                      "A, A, None) for n in (256, 1000, 4096, 9000, 20000)]",
    "moe_pack_fp4": "[L.moe_pack_fp4(A, 4, K, A, A, A, None) for K in (64, 20480)]",
    "moe_quant_rows_fp4": "[L.moe_quant_rows_fp4(A, 4, K, A, A, A, None) for K in (64, 20480)]",
    "moe_unpack_fp4": "[L.moe_unpack_fp4(moe.Fp4(A, A, A), 4, 128, A, None)]",
    "moe_linear_fp4": "[L.moe_linear_fp4(A, 128, T, N, 128, moe.Fp4(A, A, A), A, W, 1 << 30, None) "
                      "for T, N in ((1, 256), (4, 256), (100, 256), (3000, 4096))]",
}

PROGRAM = """
from ctypes import byref as i
import moe_expert_layer_sigmoid_gb300 as moe
L, A, W = moe.lib(), 1 << 21, 1 << 20
d = moe.KvDims(T=4, B=2, H=8, H_kv=2, D=128, page=16, n_pages=10, max_pages=4, max_new=0, window=0, format=1, flags=0)
st, c = moe.KvPages(A, A, A, A, A), moe.Kv(A, A, A, A, 4096, 2048, 128)
r = moe.Rope(A, None, None, 100, 64, 0, 0.0)
g = moe.RopeConfig(base=10000.0, factor=4.0, orig_len=2048.0, lo=1.0, hi=32.0, magnitude=1.0, rot=64, scaling=0)
assert {s for s in %s} == {moe.MOE_ERR_CUDA}
"""


@pytest.mark.parametrize("name", CALLS)
def test_no_device(name):
    import moe_expert_layer_sigmoid_gb300.build as b
    b.build()
    p = subprocess.run([sys.executable, "-c", PROGRAM % CALLS[name]], cwd=ROOT, env=dict(os.environ, CUDA_VISIBLE_DEVICES=""),
                       capture_output=True, text=True, timeout=300)
    assert p.returncode == 0, (p.returncode, p.stderr[-500:])
