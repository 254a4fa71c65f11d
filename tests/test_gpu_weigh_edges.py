"""Softmax weights per cached position on the GPU where rows give nothing.  Tolerances: those of test_gpu_weigh."""
import numpy as np
import pytest

from tests._util import say
from tests.test_gpu_attention4 import Batch4
from tests.test_gpu_weigh import Weights

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("cache", ["f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("seqs", [[(1, 300), (1, 40), (1, 16)], [(20, 300), (7, 90)], [(150, 400), (3, 200), (90, 90)], [(130, 700)]])
def test_rows_of_minus_infinity_give_nothing(seqs, cache):
    """Rows that the caller leaves out (a logarithm of -infinity), whatever their query holds: a padding token's may
    hold anything.  Whole tokens (not a sequence's last) and single heads, in tiles that no mask cuts, too."""
    say("rows left out", seqs, cache)
    b = Batch4(seqs, 8, 2, 64, 16, "f16", cache, seed=9)
    w, at = Weights(b), 0
    out = np.zeros((b.T, b.heads), dtype=bool)
    for n, _ in seqs:
        out[at:at + n - 1:3] = True
        out[at:at + n, 1::4] = True                          # one head of each four that share a key head
        at += n
    left = torch.from_numpy(out).cuda()
    starts = np.cumsum([0] + [n for n, _ in seqs])
    for i, h, s, _, lse in w.rows:
        s[out[starts[i]:starts[i + 1], h]] = -np.inf         # what the definition does without
    w.lse[left] = -float("inf")
    want = w.run()
    w.check(want)
    for junk in (float("nan"), float("inf")):
        b.q[left] = junk
        assert torch.equal(w.run(), want)


@pytest.mark.parametrize("n", [1, 3, 40])
def test_keys_that_are_not_finite_and_no_row(n):
    """Every row left out: new positions have 0, the others what they had, over keys of any kind."""
    say("no row", n)
    b = Batch4([(n, 200), (n, 64)], 4, 2, 64, 16, "f16", "f16", seed=3)
    w = Weights(b)
    w.lse.fill_(-float("inf"))
    for i, junk in enumerate((1.0, float("inf"), float("nan"))):
        b.tensors[0][:, :, i::5, 3] = junk
        got = w.run().cpu()
        want = w.old.cpu().clone()
        for s, (_, length) in enumerate(b.seqs):
            for j in range(length - n, length):
                want[b.table[s, j // 16].long().cpu(), :, j % 16] = 0.0
        assert torch.equal(got, want)
