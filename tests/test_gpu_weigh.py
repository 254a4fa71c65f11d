"""Softmax weights per cached position (lscd_cache_weigh) on the GPU against the plain 64-bit definition.

Tolerance, per weight, from the arithmetic (w: the sum of the rows' weights p): a row's score is off by at most
(dim + 8) 2^-24 of b = sum |scale q k| (products are exact, dim sums and the scaling round), the exponent's two
parts by 2^-22 (b + |lse|) in all (lse is an fp32 number, it and the score change units, their difference rounds),
the exponential by 2^-22; the sum of R rows and what was there before adds R 2^-24 w and 2^-23 of the result.
"""
import numpy as np
import pytest

from tests._util import say
from tests.test_gpu_attention import CHUNKS, DECODE
from tests.test_gpu_attention4 import Batch4

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L


class Weights:
    """A batch, its rows' logarithms in 64 bits, and a pool of weights."""

    def __init__(self, b, scale=None, causal=True, window=0):
        self.b, self.kw = b, dict(scale=scale, causal=causal, window=window)
        g = torch.Generator().manual_seed(5)
        self.old = torch.rand((b.pages, b.kv, b.page), generator=g).cuda()
        self.rows = []
        q, at, scale = b.q.cpu().double().numpy(), 0, b.dim ** -0.5 if scale is None else scale
        lse = np.full((b.T, b.heads), -np.inf)
        for i, (n, length) in enumerate(b.seqs):
            k, j = b.values(0, i), np.arange(length)
            p = length - n + np.arange(n)[:, None]
            seen = (j <= p if causal else j >= 0) & ((j > p - window) if window else j >= 0)
            for h in range(b.heads if n and length else 0):
                kh = k[:, h // (b.heads // b.kv)]
                s = np.where(seen, scale * (q[at:at + n, h] @ kh.T), -np.inf)
                m = np.maximum(s.max(1), -1e300)
                with np.errstate(divide="ignore"):
                    lse[at:at + n, h] = m + np.log(np.exp(s - m[:, None]).sum(1))
                self.rows.append((i, h, s, abs(scale) * (np.abs(q[at:at + n, h]) @ np.abs(kh).T), lse[at:at + n, h]))
            at += n
        self.lse = torch.from_numpy(lse).float().cuda()

    def run(self, weight=None, **more):
        b, weight = self.b, self.old.clone() if weight is None else weight
        L.lscd_cache_weigh(b.cache(), b.q, self.lse, b.start, b.length, b.table, weight, **self.kw, **more)
        torch.cuda.synchronize()
        return weight

    def check(self, got):
        b, share = self.b, self.b.heads // self.b.kv
        want, tol = self.old.cpu().double().numpy(), np.zeros(self.old.shape)
        for i, (n, length) in enumerate(b.seqs):
            if n == 0:
                continue
            w, off, seen = np.zeros((b.kv, length)), np.zeros((b.kv, length)), np.zeros((b.kv, length), dtype=bool)
            for _, h, s, big, lse in (r for r in self.rows if r[0] == i):
                on = np.isfinite(s)
                with np.errstate(invalid="ignore"):
                    p = np.where(on, np.exp(s - lse[:, None]), 0.0)
                    e = (b.dim + 8) * 2.0 ** -24 * big + 2.0 ** -22 * (big + np.abs(np.where(on, lse[:, None], 0.0)) + 1)
                w[h // share] += p.sum(0)
                off[h // share] += (p * e).sum(0) + n * share * 2.0 ** -24 * p.sum(0)
                seen[h // share] |= on.any(0)
            for j in range(length):
                at = (int(b.table[i, j // b.page]), slice(None), j % b.page)
                s = seen[:, j]
                old = want[at] * (j < length - n)
                want[at] = np.where(s, old + w[:, j], want[at])
                tol[at] = np.where(s, off[:, j] + 2.0 ** -23 * want[at] + 1e-37, 0.0)
        d = np.abs(got.cpu().double().numpy() - want)
        assert (d <= tol).all(), (int((d > tol).sum()), float((d / np.maximum(tol, 1e-300)).max()), float(d.max()))


CACHES = [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3"), ("f16", "e2m1"), ("bf16", "e2m1")]


@pytest.mark.parametrize("kind,cache", CACHES)
@pytest.mark.parametrize("heads,kv,dim,page", [(2, 2, 128, 16), (8, 2, 128, 32), (16, 1, 64, 64), (3, 3, 80, 16), (20, 1, 256, 16),
                                               (4, 4, 16, 128), (2, 2, 112, 16)])
def test_decode(heads, kv, dim, page, kind, cache):
    say(f"decode {heads}/{kv} x {dim}, page {page}, {kind} over {cache}")
    w = Weights(Batch4(DECODE, heads, kv, dim, page, kind, cache, seed=dim + heads))
    w.check(w.run())


@pytest.mark.parametrize("kind,cache", CACHES)
@pytest.mark.parametrize("heads,kv,dim,page", [(2, 2, 128, 16), (4, 1, 128, 64), (6, 2, 64, 16), (2, 2, 80, 32), (2, 1, 256, 16),
                                               (2, 2, 48, 16), (3, 1, 144, 16)])
def test_chunks(heads, kv, dim, page, kind, cache):
    say(f"chunks {heads}/{kv} x {dim}, page {page}, {kind} over {cache}")
    w = Weights(Batch4(CHUNKS, heads, kv, dim, page, kind, cache, seed=dim + heads))
    w.check(w.run())


@pytest.mark.parametrize("seqs", [[(1, 900), (1, 50), (1, 300)], [(3, 700), (2, 40)], [(200, 600), (7, 300), (1, 299)],
                                  [(4, 2), (1, 0), (3, 3)], [(1, 0)], [(200, 90), (100, 0), (5, 1)], [(700, 700)]])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 33), (True, 250), (False, 0), (False, 100)])
def test_masks(seqs, causal, window):
    """Windows, no causality, rows that see nothing: their lse is -infinity; positions that nobody sees stay."""
    say("masks", seqs, causal, window)
    w = Weights(Batch4(seqs, 4, 2, 64, 16, "f16", "f16", seed=window), causal=causal, window=window)
    w.check(w.run())


@pytest.mark.parametrize("scale", [0.0, -0.2, 2.0])
def test_scale(scale):
    say("scale", scale)
    w = Weights(Batch4([(1, 300), (40, 200)], 4, 4, 64, 16, "f16", "f16", seed=4), scale=scale)
    w.check(w.run())


def test_rows_of_one_sequence_among_idle_ones():
    """As many tokens as sequences, but all of one of them: its rows are more than one tile."""
    say("idle sequences")
    w = Weights(Batch4([(0, 30), (40, 300)] + [(0, 10)] * 40, 4, 2, 64, 16, "f16", "e4m3", seed=4))
    w.check(w.run())


def test_after_the_attention():
    """With the logarithms that the attention wrote, every row's weights sum to 1: all positions' to the rows'."""
    say("after the attention")
    for seqs in ([(1, 700), (1, 33)], [(50, 700), (3, 33), (33, 33)]):
        b = Batch4(seqs, 8, 2, 128, 16, "f16", seed=3)
        _, lse = b.run_lse()
        w = Weights(b)
        w.lse = lse
        w.old.zero_()
        got = w.run()
        for i, (n, _) in enumerate(seqs):
            pages = b.table[i][b.table[i] >= 0].long()
            total = got[pages].sum(dim=(0, 2)).cpu().double()
            # 700 weights of n x 4 rows, each off by 2^-24 of scores and logarithms of up to 64 and a few more roundings
            assert torch.allclose(total, torch.full((2,), 4.0 * n, dtype=torch.float64), rtol=2.0 ** -24 * 64 * 8, atol=0)


@pytest.mark.parametrize("cache", ["f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("seqs", [[(1, 70), (1, 16)], [(3, 50)], [(100, 230)]])
def test_garbage_where_nobody_looks(seqs, cache):
    """Keys that are not finite behind the last position, before the window and in spare pages; what is not seen
    keeps its weight, NaN or not; new tokens' positions take theirs over NaN."""
    say("garbage", seqs, cache)
    b = Batch4(seqs, 4, 2, 64, 32, "f16", cache, seed=2)
    w = Weights(b, window=40)
    clean = w.run()
    w.check(clean)
    used, new = (torch.zeros((b.pages, b.page), dtype=torch.bool) for _ in range(2))
    for i, (n, length) in enumerate(seqs):
        for j in range(length):
            at = (b.table[i, j // 32].long(), j % 32)
            used[at], new[at] = j > length - n - 40, j >= length - n
    which = 2 if cache == "e2m1" else 0
    x = b.tensors[which].view(torch.uint8 if cache != "f16" else torch.int16)
    x[~used[:, None].expand(-1, 2, -1).cuda()] = 255 if cache == "e2m1" else 127 if cache == "e4m3" else 0x7E00
    hole = ~used | new
    old = torch.where(hole[:, None].cuda(), torch.full_like(w.old, float("nan")), w.old)
    got = w.run(old.clone())
    seen = used[:, None].expand(-1, 2, -1).cuda()
    assert torch.equal(got[seen], clean[seen]) and torch.isnan(got[~seen]).all()


def test_later_tokens_do_not_count_for_earlier_rows():
    """A key that is not a number in new token j: weights of the tokens before it come from the rows that do not see it."""
    say("later tokens")
    b = Batch4([(60, 150)], 2, 2, 64, 16, "f16", "f16", seed=8)
    w = Weights(b)
    clean = w.run()
    at = 150 - 1                                             # the last token: its row alone sees it
    b.tensors[0][b.table[0, at // 16].long(), :, at % 16, 5] = float("inf")
    bad = w.run()
    sees = torch.zeros((b.pages, 16), dtype=torch.bool)
    sees[b.table[0, at // 16].long().cpu(), at % 16] = True
    rest = ~sees[:, None].expand(-1, 2, -1).cuda()
    assert torch.equal(bad[rest], clean[rest]) and not torch.equal(bad[~rest], clean[~rest])


def test_twice_adds_and_is_the_same():
    say("twice")
    for seqs in (DECODE, CHUNKS):
        b = Batch4(seqs, 4, 2, 64, 16, "bf16", "e4m3", seed=1)
        w = Weights(b)
        one = w.run()
        for _ in range(3):
            assert torch.equal(w.run(), one)
        zero = Weights(b)
        zero.old.zero_()
        alone = zero.run()
        two = w.run(one.clone())
        old = torch.zeros_like(one, dtype=torch.bool)
        for i, (n, length) in enumerate(seqs):
            for j in range(length - n if n else 0):
                old[b.table[i, j // 16].long(), :, j % 16] = True
        assert torch.equal(two[~old], one[~old]) and torch.equal(two[old], (one + alone)[old])


def test_offsets_past_32_bits():
    """Weights at the end of a pool of more than 2^32 bytes of them, keys past 2^31 bytes."""
    say("large pool")
    b = Batch4([(1, 100), (30, 90)], 8, 8, 16, 16, "f16", "e2m1", seed=12)
    pages = (2 ** 30 + 2 ** 26) // (8 * 16)
    w = Weights(b)
    small = w.run()
    w.check(small)
    at = pages - b.pages
    big = [torch.empty((pages, *x.shape[1:]), dtype=torch.uint8, device="cuda") for x in b.tensors]
    for x, y in zip(big, b.tensors):
        x[at:] = y
    weight = torch.zeros((pages, 8, 16), device="cuda")
    weight[at:] = w.old
    b.tensors, b.table = big, torch.where(b.table < 0, b.table, b.table + at).to(torch.int32)
    w.run(weight)
    assert torch.equal(weight[at:], small) and not weight[:at].any()


def test_contents_out_of_range_are_clamped():
    """Lengths past the table, pages outside the pool (no weight), starts past T."""
    say("clamped contents")
    for n in (1, 50):
        b = Batch4([(n, 60), (n, 30)], 4, 2, 64, 16, "f16", "f16", seed=3)
        w = Weights(b)
        b.table[1, 0] = 2 ** 30
        got = w.run()
        kept = torch.ones(b.pages, dtype=torch.bool)
        for p in list(b.table[0, :4]) + [b.table[1, 1]]:
            kept[int(p)] = False
        assert torch.equal(got[kept.cuda()], w.old[kept.cuda()])
        b.length[0] = 2 ** 30
        b.start[2] = 2 ** 30
        assert w.run().shape == w.old.shape


def test_strides_stream_and_graph():
    say("strides, stream, graph")
    for seqs in ([(1, 300), (1, 20)], [(40, 300), (1, 20), (3, 64)]):
        b = Batch4(seqs, 4, 2, 64, 16, "f16", "e2m1", seed=11)
        w = Weights(b)
        want = w.run()
        wide = torch.full((b.T, 3, 4, 64), 5.0, dtype=torch.float16, device="cuda")
        wide[:, 1] = b.q
        weight, cache = w.old.clone(), b.cache()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.lscd_cache_weigh(cache, wide[:, 1], w.lse, b.start, b.length, b.table, weight)
        s.synchronize()
        assert torch.equal(weight, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lscd_cache_weigh(cache, b.q, w.lse, b.start, b.length, b.table, weight)
        for k in range(4):
            b.length.copy_(torch.tensor([n - 3 * k for _, n in seqs], dtype=torch.int32))
            b.q.normal_()
            weight.copy_(w.old)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(weight, w.run())


def test_nothing_to_do_and_refusals():
    say("refusals")
    b = Batch4([(1, 60), (20, 90)], 4, 2, 64, 16, "f16", "f16")
    w, c = Weights(b), b.cache()
    before = w.old.clone()
    L.lscd_cache_weigh(c, b.q[:0], w.lse[:0], b.start * 0, b.length, b.table, w.old)
    L.lscd_cache_weigh(c, b.q, w.lse, b.start[:1], b.length[:0], b.table[:0], w.old)
    L.lscd_cache_weigh(c, b.q, w.lse, b.start * 0, b.length, b.table, w.old)
    assert torch.equal(w.old, before)
    good = (c, b.q, w.lse, b.start, b.length, b.table, w.old)

    def put(i, x):
        return (*good[:i], x, *good[i + 1:])

    for args in (put(1, b.q.float()), put(1, b.q[:, :, :32]), put(2, w.lse[:-1]), put(2, w.lse.half()), put(3, b.start[:-1]),
                 put(4, b.length.long()), put(5, b.table[:1]), put(6, w.old[:-1]), put(6, w.old.double()),
                 put(6, w.old.transpose(1, 2)), put(6, w.old.cpu())):
        with pytest.raises(ValueError):
            L.lscd_cache_weigh(*args)

    def status(*args, **kw):
        with pytest.raises(L.LSCDError) as e:
            L.lscd_cache_weigh(*args, **kw)
        return e.value.status

    assert status(*put(1, b.q.bfloat16())) == L.LSCD_ERROR_NOT_SUPPORTED
    assert status(*good, scale=float("inf")) == L.LSCD_ERROR_INVALID_VALUE
    assert status(*good, window=-1) == L.LSCD_ERROR_INVALID_VALUE
    three = b.q[:, :3].contiguous()                          # not a multiple of the cache's two heads
    assert status(c, three, w.lse[:, :3].contiguous(), *good[3:]) == L.LSCD_ERROR_INVALID_VALUE
    assert torch.equal(w.old, before)


def test_many_sequences():
    """More than 64 sequences of both kinds, idle ones among them, in one call."""
    say("many sequences")
    seqs = [(i % 3, 20 + 7 * i % 90) for i in range(70)] + [(45, 200), (0, 0), (1, 300)] + [(i % 2, 33 + i) for i in range(60)] + [(90, 90)]
    w = Weights(Batch4(seqs, 4, 1, 64, 16, "f16", "e2m1", seed=2))
    w.check(w.run())


@pytest.mark.parametrize("n", [0, 1, 9, 33])
def test_one_sequence_with_room_for_more(n):
    """A captured call's room: 40 rows of 4 heads in q, fewer new tokens in `start`; rows behind them do not count."""
    say("room", n)
    b = Batch4([(n, 150)], 4, 1, 64, 16, "f16", "f16", seed=3)
    w = Weights(b)
    want = w.run()
    w.check(want)
    b.q = torch.cat([b.q, torch.full((40 - n, 4, 64), float("nan"), device="cuda").half()])
    w.lse = torch.cat([w.lse, torch.zeros((40 - n, 4), device="cuda")])
    got = w.run()
    # (another kernel may serve it: the sums' order differs)
    assert torch.allclose(got, want, rtol=2.0 ** -18, atol=1e-9)


@pytest.mark.parametrize("n", [1, 100])
def test_keys_past_the_largest_count_as_the_largest(n):
    """As in the attention: a key's 65536 is 65504, so that a query of zeros there sees zero."""
    say("largest keys", n)
    b = Batch4([(n, 70)], 2, 2, 64, 16, "f16", "e2m1", seed=5)
    b.q[:, :, 32:] = 0
    clean = Weights(b)
    want = clean.run()
    b.tensors[2][..., 1] = 127 + 14
    b.tensors[0][..., 16:] = 0x77
    got = clean.run()
    assert torch.isfinite(got).all() and torch.equal(got, want)
