"""The decoder block example: chunked prefill and decode through the cache give what the whole
sequences give."""
import os
import sys

import pytest

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.mark.parametrize("fmt", ["bf16", "e4m3", "int4"])
def test_decoder_block(fmt):
    import decoder_block
    off, same, moved = decoder_block.main(fmt)
    # x is the same in both runs, so the projections are too up to the shape-dependent order of a
    # product's sum, which can move a bf16 key or value by its last bit (2^-8), and a code of four
    # bits by one of its 15 steps; weights and outputs round to bf16 on top
    assert off < (0.1 if fmt == "bf16" else 0.5)
    # a moved key may tip a router's choice between two near-equal experts for a token
    assert moved < 0.2
