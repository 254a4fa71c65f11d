"""Eviction from a paged cache on the GPU: the memory of the positions kept, on another stream than the current one."""
import numpy as np
import pytest

from tests._util import say
from tests.test_gpu_evict import Pool

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L


@pytest.mark.parametrize("raw", [False, True])
@pytest.mark.parametrize("to", [False, True])
def test_positions_kept_belong_to_the_calls_stream(raw, to):
    """On another stream the tensor that the call allocates is that stream's: not a block that the current stream has
    just given back (its work may still use it), and not one that the current stream gets next (the call's may)."""
    say("kept on another stream", raw, to)
    keep = 2048                                              # (3 x 2 x 2048 numbers: 48 KB, rounded to 512 bytes)
    p = Pool([3000, 2100, 2500], keep, 2, 16, 64, "f16", seed=6)
    cache, shape, to_table = p.device(), (3, 2, keep), p.to.cuda() if to else None
    want = p.expect(9, to)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    mine = torch.empty(shape, dtype=torch.int32, device="cuda")
    was = mine.data_ptr()
    del mine
    kept = L.lscd_cache_evict(cache, p.w, *p.args, keep, 9, to=to_table, stream=s.cuda_stream if raw else s)
    at = kept.data_ptr()
    assert at != was
    s.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[0])
    assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(p.bytes, want[1]))
    del kept
    others = [torch.empty(shape, dtype=torch.int32, device="cuda") for _ in range(4)]
    assert at not in [x.data_ptr() for x in others]


def test_a_result_that_nobody_keeps():
    """The returned tensor dropped, and its size allocated and overwritten at once on the current stream."""
    say("result dropped")
    p = Pool([3000, 2100, 2500], 2048, 2, 16, 64, "e4m3", seed=7)
    want = p.expect(0, False)
    s = torch.cuda.Stream()
    for _ in range(3):
        cache = p.device()
        s.wait_stream(torch.cuda.current_stream())
        L.lscd_cache_evict(cache, p.w, *p.args, 2048, stream=s)
        junk = [torch.full((3, 2, 2048), 5, dtype=torch.int32, device="cuda") for _ in range(4)]
        s.synchronize()
        assert len(junk) == 4 and all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(p.bytes, want[1]))


def stream_of(t):
    """The stream whose pool a tensor's memory is of."""
    for s in torch.cuda.memory_snapshot():
        if s["address"] <= t.data_ptr() < s["address"] + s["total_size"]:
            return s["stream"]


def test_every_way_to_name_a_stream():
    """None, a stream, its handle, and the default stream's, which is 0: from under another current stream."""
    say("ways to name a stream")
    p, s, other = Pool([300], 64, 2, 16, 16, "f16", seed=1), torch.cuda.Stream(), torch.cuda.Stream()
    want = p.expect(3, True)[0]
    assert stream_of(torch.empty(5, device="cuda")) == torch.cuda.current_stream().cuda_stream == 0
    for stream, handle in ((None, other.cuda_stream), (s, s.cuda_stream), (s.cuda_stream, s.cuda_stream), (0, 0),
                           (torch.cuda.default_stream(), 0)):
        cache, to = p.device(), p.to.cuda()
        torch.cuda.synchronize()
        with torch.cuda.stream(other):
            kept = L.lscd_cache_evict(cache, p.w, *p.args, 64, 3, to=to, stream=stream)
        torch.cuda.synchronize()
        assert stream_of(kept) == handle and np.array_equal(kept.cpu().numpy(), want)
