"""The paged cache at the ends of its arguments: slots named twice, calls of more tokens than one launch takes."""
import numpy as np
import pytest

from tests._util import say
from tests.test_gpu_cache import expect_write, host, pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L


@pytest.mark.parametrize("dim", [64, 80])
def test_a_slot_named_twice_leaves_the_others(dim):
    """What such a slot holds is undefined; every other slot, next to it or not, holds what it should."""
    say("a slot named twice", dim)
    T, heads, page, pages = 60, 5, 16, 6
    c = pool(pages, heads, page, dim, "e4m3", 3)
    before = [host(x) for x in c]
    rng = np.random.default_rng(dim)
    x = torch.from_numpy(rng.standard_normal((T, heads, dim)) * np.exp(3 * rng.standard_normal((T, heads, 1)))).half().cuda()
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[40], slots[41], slots[59] = slots[3], slots[39], slots[0]
    L.lscd_cache_write(L.Cache(*c), x, -x, torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    once = np.ones(pages * page, dtype=bool)
    once[slots[[0, 3, 39]]] = False
    once = once.reshape(pages, page)
    for i in range(2):
        codes, scales = expect_write((x if i == 0 else -x).cpu().double().numpy(), slots, before[i], before[2 + i], page)
        assert np.array_equal(host(c[i]).transpose(0, 2, 1, 3)[once], codes.transpose(0, 2, 1, 3)[once])
        assert np.array_equal(host(c[2 + i]).transpose(0, 2, 1)[once], scales.transpose(0, 2, 1)[once])


@pytest.mark.parametrize("T", [2 ** 28 + 40, 2 ** 29 + 40])
def test_more_tokens_than_a_launch_takes(T):
    """The last tokens of a call of more than 2^28 and 2^29 are written and read like the first."""
    say("many tokens", T)
    c = [torch.zeros((3, 1, 16, 16), dtype=torch.float16, device="cuda") for _ in range(2)]
    cache = L.Cache(*c)
    x = torch.empty((T, 1, 16), dtype=torch.float16, device="cuda")
    slots = torch.full((T,), -1, dtype=torch.int32, device="cuda")
    at = [0, 2 ** 28 - 1, 2 ** 28, T // 2, T - 2, T - 1]
    for i, t in enumerate(at):
        x[t], slots[t] = i + 1, 5 * i
    L.lscd_cache_write(cache, x, x, slots)
    want = torch.zeros((48,))
    want[torch.arange(len(at)) * 5] = torch.arange(len(at)) + 1.0
    for k in c:
        assert torch.equal(k.cpu().float(), want.view(3, 1, 16, 1).expand(3, 1, 16, 16))
    x.fill_(7)
    L.lscd_cache_read(cache, slots, x, x)
    for i, t in enumerate(at):
        assert (x[t] == i + 1).all()
    assert (x[T - 3] == 0).all() and (x[1] == 0).all()
