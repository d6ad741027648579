"""Weights in parts: rows of a packed matrix from a multiple of 128 on are weights of their own, without a copy."""
import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("T", [1, 2, 5, 40, 100, 300, 2000])
@pytest.mark.parametrize("N,K,cuts", [(520, 192, [0, 128, 384, 520]), (2056, 1024, [0, 1024, 2056]), (12288, 448, [0, 8192, 12288])])
def test_parts(T, N, K, cuts):
    g = torch.Generator().manual_seed(T + N)
    x = torch.randn(T, K, generator=g).to(torch.bfloat16).cuda()
    q, b, s = moe.moe_pack_fp4(torch.randn(N, K, generator=g).cuda())
    ws = moe.workspace(moe.moe_linear_fp4_workspace_bytes(T, N, K))
    whole = torch.empty(T, N, dtype=torch.bfloat16, device="cuda")
    moe.moe_linear_fp4(x, moe.fp4(q, b, s), whole, ws)
    tile = K // 64 * 512
    for lo, hi in zip(cuts, cuts[1:]):
        end = lo // 128 * tile + moe.moe_fp4_scale_bytes(hi - lo, K)
        w = moe.fp4(q[lo:hi], b[lo // 128 * tile:end], s[lo:hi])
        out = torch.empty(T, hi - lo, dtype=torch.bfloat16, device="cuda")
        moe.moe_linear_fp4(x, w, out, ws)
        assert moe.moe_check_device_status(ws) == moe.MOE_OK
        # sums of other cuts of K, or of another kernel, differ in their last bits: by a rounding of bf16 and what cancels
        size = (moe.moe_unpack_fp4(*moe.moe_quant_rows_fp4(x)).double().abs() @ moe.moe_unpack_fp4(q[lo:hi], b[lo // 128 * tile:end], s[lo:hi]).double().abs().T)
        room = 2.0 ** -7 * whole[:, lo:hi].double().abs() + (K + 8) * 2.0 ** -22 * 1.01 * size
        assert ((out.double() - whole[:, lo:hi].double()).abs() <= room).all()
