"""The attention's factor of the scores: what is refused on the host."""
import pytest

from test_kv_attn_host import INV, L, _attn  # noqa: F401  (L: the fixture)


@pytest.mark.parametrize("scale", [float("inf"), -float("inf"), float("nan"), 3.0e38, -2.4e38, 3.4e38])
def test_factors_without_an_exponent(L, scale):  # noqa: F811
    """e^(scale * s) is taken as a power of two: a factor whose product with log2(e) overflows is none."""
    assert _attn(L, scale=scale) == INV
