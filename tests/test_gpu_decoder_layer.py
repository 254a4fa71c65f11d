"""The example's decoder layer: a prompt and decoded tokens through all serving operators and the
sparse product, against the same layer in float32 without a cache.

The difference is dominated by the cache's 8-bit values: e4m3 rounds keys and values by up to 2^-4
relative (a uniform error of rms 2^-4 / sqrt(3), smaller for most fractions); averaged over the tokens
that a row sees and added to the residual stream, it has to stay well under 2^-4 of the output.
"""
import os
import sys

import pytest

from tests._util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("hidden,heads,prompts", [(512, 4, [37, 1, 20]), (1024, 16, [90, 64])])
def test_decoder_layer(hidden, heads, prompts):
    say("decoder layer", hidden, heads, prompts)
    sys.path.insert(0, os.path.join(ROOT, "examples"))
    try:
        import decoder_layer as ex
    finally:
        sys.path.pop(0)
    layer = ex.Layer(hidden, heads, pages=64)
    xs, ys, _ = ex.serve(layer, prompts, 5)
    want = layer.plain(torch.cat(xs), [len(v) for v in xs])
    got = torch.cat(ys).float()
    assert got.shape == want.shape and torch.isfinite(got).all()
    assert float((got - want).norm() / want.norm()) < 2.0 ** -4 / 3 ** 0.5
