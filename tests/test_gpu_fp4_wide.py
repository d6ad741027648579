"""Projections of 65 to 128 tokens on weights of many rows: a pair's tile is half empty, and rows behind the last stay."""
import math

import pytest
import torch

import moe_expert_layer_sigmoid_gb300 as moe
from test_gpu_fp4 import check, project, rows_of

pytestmark = pytest.mark.gpu


# either side of as many wide tiles as SMs (152 of 128 rows: 19456)
@pytest.mark.parametrize("T,N,K", [
    (65, 19456, 128), (65, 19464, 64), (127, 19464, 448), (128, 19456, 1344), (128, 19592, 1088), (100, 20000, 2624), (66, 40008, 576),
    (128, 32768, 256),
])
def test_projection_of_few_tokens_on_many_rows(T, N, K):
    g = torch.Generator().manual_seed(T + N + K)
    x = rows_of(T, K, "outliers", seed=T).to(torch.bfloat16)
    w = torch.randn(N, K, generator=g) / math.sqrt(K)
    buf = torch.full((T + 130, N), 7.0, dtype=torch.bfloat16, device="cuda")
    check(project(x.cuda(), w, T, N, K, out=buf[:T]), x, w)
    assert (buf[T:] == 7).all()
