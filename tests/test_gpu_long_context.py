"""The operators for long contexts together, as a decoder layer uses them (examples/decoder_layer.py): a prompt and
captured decoding over a 4-bit cache, prompts cut by the weights of their attention.

The 4-bit cache's part of the difference from a plain layer: e2m1 rounds keys and values by up to 2^-2 relative (a
uniform error of rms 2^-2 / sqrt(3), smaller for most); averaged over the tokens that a row sees and added to the
residual stream, it has to stay under that, as the 8-bit cache's under 2^-4 / sqrt(3).
"""
import os
import sys

import pytest

from tests._util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))
try:
    if torch.cuda.is_available():
        import decoder_layer as ex
finally:
    sys.path.pop(0)


@pytest.mark.parametrize("hidden,heads,prompts", [(512, 4, [37, 1, 20]), (1024, 16, [90, 64]), (640, 8, [50, 33])])
def test_decoder_layer_over_a_4_bit_cache(hidden, heads, prompts):
    say("decoder layer, 4 bits", hidden, heads, prompts)
    layer = ex.Layer(hidden, heads, pages=64, cache="e2m1")
    xs, ys, _ = ex.serve(layer, prompts, 5)
    want = layer.plain(torch.cat(xs), [len(v) for v in xs])
    got = torch.cat(ys).float()
    assert got.shape == want.shape and torch.isfinite(got).all()
    assert float((got - want).norm() / want.norm()) < 2.0 ** -2 / 3 ** 0.5


@pytest.mark.parametrize("cache", ["e4m3", "e2m1"])
def test_keeping_everything_changes_nothing(cache):
    say("keep everything", cache)
    prompts = [37, 90, 1]
    one = ex.serve(ex.Layer(512, 4, pages=64, cache=cache), prompts, 4)[1]
    two = ex.serve(ex.Layer(512, 4, pages=64, cache=cache), prompts, 4, keep=90)[1]
    assert all(torch.equal(a, b) for a, b in zip(one, two))


@pytest.mark.parametrize("cache", ["e4m3", "e2m1"])
def test_cut_prompts_go_on(cache):
    """Sequences that are short enough decode as before; the others from what is kept, and each step's graph replays."""
    say("cut prompts", cache)
    prompts = [37, 200, 16]
    layer = ex.Layer(512, 4, pages=64, cache=cache)
    whole = ex.serve(ex.Layer(512, 4, pages=64, cache=cache), prompts, 6)[1]
    cut = ex.serve(layer, prompts, 6, keep=64)[1]
    assert all(torch.isfinite(y).all() and y.shape == z.shape for y, z in zip(cut, whole))
    assert torch.equal(cut[0][:37], whole[0][:37]) and torch.equal(cut[1][:200], whole[1][:200])
    # (another length of one sequence moves where the work of the others is split: the last bits may differ)
    for s in (0, 2):
        assert float((cut[s] - whole[s]).float().norm() / whole[s].float().norm()) < 2.0 ** -10
    assert not torch.equal(cut[1][200:], whole[1][200:])
