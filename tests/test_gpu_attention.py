"""Attention over a paged cache on the GPU against the plain 64-bit definition.

Tolerance, per value, from the arithmetic (u: unit roundoff of the type, A = sum_j p_j |v_j|):
  u |o|          the output's rounding;
  (u + e) A      the weights' rounding to the type, and e for everything in fp32: scores off by
                 at most (dim + 8) 2^-24 of sum |scale q k|, which enters numerator and denominator,
                 and 2^-18 for exponentials and the sums' orders;
  tiny * len     weights below the type's normal range, times the largest |v|.
"""
import numpy as np
import pytest

from oracle import serving as sv
from tests._util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L

TYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


class Batch:
    """Sequences of given (new tokens, length) in a shuffled pool; the values beside it in 64 bits."""

    def __init__(self, seqs, heads, kv, dim, page, kind, cache, seed=0, spare=2):
        g = torch.Generator().manual_seed(seed)
        self.seqs, self.heads, self.kv, self.dim, self.page, self.kind = seqs, heads, kv, dim, page, kind
        need = [(n + page - 1) // page for _, n in seqs]
        self.pages = sum(need) + spare
        shape = (self.pages, kv, page, dim)
        if cache == "e4m3":
            codes = [(torch.randn(shape, generator=g) * 60).clamp(-448, 448).to(torch.float8_e4m3fn) for _ in range(2)]
            scales = [torch.exp2(torch.randint(-8, -4, shape[:3], generator=g).float()) for _ in range(2)]
            self.tensors = [x.cuda() for x in codes + scales]
        else:
            self.tensors = [torch.randn(shape, generator=g).to(TYPES[kind]).cuda() for _ in range(2)]
        self.table = torch.full((max(1, len(seqs)), max(need + [1]) + 1), -1, dtype=torch.int32)
        order, at = torch.randperm(self.pages, generator=g).to(torch.int32), 0
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
        self.table = self.table[:len(seqs)].cuda()
        self.start = torch.tensor(np.concatenate([[0], np.cumsum([n for n, _ in seqs])]), dtype=torch.int32, device="cuda")
        self.length = torch.tensor([n for _, n in seqs], dtype=torch.int32, device="cuda")
        self.T = sum(n for n, _ in seqs)
        self.q = (torch.randn((self.T, heads, dim), generator=g) * 1.5).to(TYPES[kind]).cuda()
        self.handle = L.lscd_attention_create(heads, kv, dim)

    def cache(self):
        return L.Cache(*self.tensors)

    def run(self, q=None, out=None, **kw):
        q = self.q if q is None else q
        out = torch.full_like(self.q, float("nan")) if out is None else out
        L.lscd_attention(self.handle, self.cache(), q, self.start, self.length, self.table, out, **kw)
        torch.cuda.synchronize()
        return out

    def values(self, which, i):
        x = self.tensors[which].double() if len(self.tensors) == 2 else \
            self.tensors[which].double() * self.tensors[2 + which].double()[..., None]
        n = self.seqs[i][1]
        pages = self.table[i, :(n + self.page - 1) // self.page].long()
        return x[pages].permute(0, 2, 1, 3).reshape(-1, self.kv, self.dim)[:n].cpu().numpy()

    def check(self, out, q=None, scale=None, causal=True, window=0):
        q = (self.q if q is None else q).cpu().double().numpy()
        scale = self.dim ** -0.5 if scale is None else scale
        u, at, got = sv.ROUNDOFF[self.kind], 0, out.cpu().double().numpy()
        for i, (n, length) in enumerate(self.seqs):
            o, a, big = sv.attention(q[at:at + n], self.values(0, i), self.values(1, i), scale, causal, window)
            e = 2 * (self.dim + 8) * 2.0 ** -24 * big[..., None] + 2.0 ** -18
            top = np.abs(self.values(1, i)).max() if length else 0.0
            tol = u * np.abs(o) + (u + e) * a + sv.TINY[self.kind] * (1 + length * top)
            d = np.abs(got[at:at + n] - o)
            assert d.shape == o.shape and (d <= tol).all(), (i, n, length, float((d / np.maximum(tol, 1e-300)).max()))
            at += n


DECODE = [(1, 1), (1, 2), (1, 31), (1, 33), (1, 128), (1, 129), (1, 517), (0, 40), (1, 1000)]
CHUNKS = [(5, 5), (130, 130), (64, 400), (0, 0), (1, 77), (33, 300), (257, 513)]


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("heads,kv,dim,page", [(2, 2, 128, 16), (8, 2, 128, 32), (16, 1, 64, 64), (3, 3, 80, 16), (20, 1, 256, 16),
                                               (4, 4, 16, 128)])
def test_decode(heads, kv, dim, page, kind, cache):
    say(f"decode {heads}/{kv} x {dim}, page {page}, {kind} over {cache}")
    b = Batch(DECODE, heads, kv, dim, page, kind, cache, seed=dim + heads)
    b.check(b.run())


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("heads,kv,dim,page", [(2, 2, 128, 16), (4, 1, 128, 64), (6, 2, 64, 16), (2, 2, 80, 32), (2, 1, 256, 16)])
def test_chunks(heads, kv, dim, page, kind, cache):
    say(f"chunks {heads}/{kv} x {dim}, page {page}, {kind} over {cache}")
    b = Batch(CHUNKS, heads, kv, dim, page, kind, cache, seed=dim + heads)
    b.check(b.run())


@pytest.mark.parametrize("seqs", [[(1, 900), (1, 50), (1, 300)], [(3, 700), (2, 40)], [(200, 600), (7, 300), (1, 299)]])
@pytest.mark.parametrize("causal,window", [(True, 1), (True, 33), (True, 250), (False, 0), (False, 100)])
def test_masks(seqs, causal, window):
    say("masks", seqs, causal, window)
    b = Batch(seqs, 4, 2, 64, 16, "f16", "f16", seed=window)
    b.check(b.run(causal=causal, window=window), causal=causal, window=window)


@pytest.mark.parametrize("seqs", [[(4, 2), (1, 0), (3, 3)], [(1, 0)], [(200, 90), (100, 0), (5, 1)]])
def test_rows_that_see_nothing(seqs):
    """More new tokens than positions: the first tokens stand before the cache and see nothing."""
    say("empty rows", seqs)
    b = Batch(seqs, 4, 2, 128, 16, "f16", "f16")
    out = b.run()
    b.check(out)
    assert (out[:max(0, seqs[0][0] - seqs[0][1])] == 0).all()
    if seqs[0][0] > 1:
        b.check(b.run(causal=False, window=3), causal=False, window=3)


@pytest.mark.parametrize("scale", [0.0, -0.2, 1.0])
def test_scale(scale):
    say("scale", scale)
    b = Batch([(1, 300), (40, 200)], 4, 4, 64, 16, "f16", "f16", seed=4)
    b.check(b.run(scale=scale), scale=scale)


def test_large_scores():
    """Scores that climb along the positions by hundreds: the maximum moves again and again."""
    say("large scores")
    for kind in ("f16", "bf16"):
        b = Batch([(1, 700), (150, 700)], 2, 2, 64, 16, kind, kind, seed=8)
        b.q.fill_(1.0)
        k = b.tensors[0]
        for i in range(2):
            for j in range(700):
                k[b.table[i, j // 16].long(), :, j % 16] = (j % 350) / 350 * (1 if i else 2)
        b.check(b.run(scale=4.0), scale=4.0)


@pytest.mark.parametrize("cache", ["f16", "e4m3"])
@pytest.mark.parametrize("seqs", [[(1, 70), (1, 16)], [(3, 50)], [(100, 230)]])
def test_garbage_where_nobody_looks(seqs, cache):
    """NaN and infinities in spare pages, behind the last position, in later tokens and before the window."""
    say("garbage", seqs, cache)
    b = Batch(seqs, 4, 2, 64, 32, "f16", cache, seed=2)
    clean = b.run(window=40)
    b.check(clean, window=40)
    used = torch.zeros((b.pages, b.page), dtype=torch.bool)
    for i, (n, length) in enumerate(seqs):
        for j in range(length):
            if j > length - n - 40:
                used[b.table[i, j // 32].long(), j % 32] = True
    for x in b.tensors[:2]:
        bad = torch.full(x.shape, float("nan")).to(x.dtype).cuda()
        keep = used[:, None, :, None].cuda()
        x.view(torch.uint8 if cache == "e4m3" else torch.int16).copy_(torch.where(
            keep, x.view(torch.uint8 if cache == "e4m3" else torch.int16), bad.view(torch.uint8 if cache == "e4m3" else torch.int16)))
    assert torch.equal(b.run(window=40), clean)


@pytest.mark.parametrize("n,heads", [(4, 4), (100, 2), (7, 2)])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_later_tokens_do_not_reach_earlier_ones(n, heads, bad):
    """A value that is not finite in new token j reaches tokens j.. only; the same before a window."""
    say("later tokens", n, bad)
    length, page = 150, 16
    b = Batch([(n, length)], heads, 2, 64, page, "f16", "f16", seed=n)
    clean = b.run()
    j = n // 2
    at = length - n + j
    slot = (b.table[0, at // page].long(), slice(None), at % page)
    for which in (0, 1):
        keep = b.tensors[which][slot].clone()
        b.tensors[which][slot[0], :, slot[2], 3] = bad
        out = b.run()
        assert torch.equal(out[:j], clean[:j]), which
        if which == 1:
            assert not torch.isfinite(out[j:, :, 3]).any()
            assert torch.equal(out[j:, :, 4:], clean[j:, :, 4:])
        windowed = b.run(window=1)                           # token i sees position at - j + i only
        assert torch.isfinite(windowed[torch.arange(n) != j]).all()
        b.tensors[which][slot] = keep


def test_one_long_sequence_and_many_short_ones():
    """Work is cut inside the long one; every part arrives, whatever the others are; twice the same."""
    say("long and short")
    seqs = [(1, 6000)] + [(1, 1 + 37 * i % 200) for i in range(130)]
    b = Batch(seqs, 4, 2, 64, 16, "f16", "e4m3", seed=1)
    one = b.run()
    b.check(one)
    for _ in range(3):
        assert torch.equal(b.run(), one)
    seqs = [(300, 3000), (1, 50), (40, 40)]
    b = Batch(seqs, 4, 1, 128, 64, "bf16", "bf16", seed=1)
    one = b.run()
    b.check(one)
    for _ in range(3):
        assert torch.equal(b.run(), one)


def test_strides():
    """q, out and the table as slices of wider tensors."""
    say("strides")
    b = Batch([(1, 60), (20, 90)], 4, 2, 64, 16, "f16", "f16", seed=6)
    wide = torch.full((b.T, 3, 4, 64), 5.0, dtype=torch.float16, device="cuda")
    wide[:, 1] = b.q
    table = torch.full((2, b.table.shape[1] + 5), 9, dtype=torch.int32, device="cuda")
    table[:, :b.table.shape[1]] = b.table
    b.table = table[:, :b.table.shape[1]]
    out = b.run(q=wide[:, 1], out=wide[:, 2])
    b.check(out)
    assert (wide[:, 0] == 5).all() and torch.equal(wide[:, 1], b.q)


def test_offsets_past_32_bits():
    """Pages at the end of a pool of more than 2^31 values."""
    say("large pool")
    b = Batch([(1, 100), (30, 90)], 8, 8, 128, 16, "f16", "f16", seed=12)
    pages = (2 ** 31 + 2 ** 27) // (8 * 16 * 128)
    big = [torch.empty((pages, 8, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    for x, y in zip(big, b.tensors):
        x[pages - b.pages:] = y
    small = b.run()
    b.check(small)
    b.tensors, b.table = big, torch.where(b.table < 0, b.table, b.table + (pages - b.pages)).to(torch.int32)
    assert torch.equal(b.run(), small)


def test_contents_out_of_range_are_clamped():
    """Lengths past the table, pages outside the pool, starts past T: no access out of bounds, no error."""
    say("clamped contents")
    for n in (1, 50):
        b = Batch([(n, 60), (n, 30)], 4, 2, 64, 16, "f16", "f16", seed=3)
        b.length[0] = 2 ** 30
        b.table[1, 0] = 2 ** 30
        b.start[2] = 2 ** 30
        out = b.run()
        assert out.shape[0] == 2 * n


def test_stream_and_graph():
    """On another stream; captured once and replayed with other lengths and queries."""
    say("stream, graph")
    for seqs in ([(1, 300), (1, 20)], [(40, 300), (1, 20), (3, 64)]):
        b = Batch(seqs, 4, 2, 64, 16, "f16", "f16", seed=11)
        want = b.run()
        out = torch.empty_like(want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.lscd_attention(b.handle, b.cache(), b.q, b.start, b.length, b.table, out)
        s.synchronize()
        assert torch.equal(out, want)
        cache = b.cache()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lscd_attention(b.handle, cache, b.q, b.start, b.length, b.table, out)
        for k in range(4):
            b.length.copy_(torch.tensor([n - 3 * k for _, n in seqs], dtype=torch.int32))
            b.q.normal_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, b.run())


def test_nothing_to_do_and_refusals():
    say("refusals")
    b = Batch([(1, 60), (20, 90)], 4, 2, 64, 16, "f16", "f16")
    c = b.cache()
    L.lscd_attention(b.handle, c, b.q[:0], b.start * 0, b.length, b.table, b.q[:0])
    L.lscd_attention(b.handle, c, b.q, b.start[:1], b.length[:0], b.table[:0], torch.empty_like(b.q))

    def status(*args, **kw):
        with pytest.raises(L.LSCDError) as e:
            L.lscd_attention(*args, **kw)
        return e.value.status

    out = torch.empty_like(b.q)
    with pytest.raises(ValueError):
        L.lscd_attention(b.handle, c, b.q, b.start[:-1], b.length, b.table, out)
    with pytest.raises(ValueError):
        L.lscd_attention(b.handle, c, b.q, b.start, b.length, b.table.long(), out)
    with pytest.raises(ValueError):
        L.lscd_attention(b.handle, c, b.q, b.start, b.length, b.table, out.bfloat16())
    with pytest.raises(ValueError):
        L.lscd_attention(b.handle, c, b.q[:, :2], b.start, b.length, b.table, out)
    assert status(b.handle, c, b.q.bfloat16(), b.start, b.length, b.table, out.bfloat16()) == L.LSCD_ERROR_NOT_SUPPORTED
    assert status(b.handle, c, b.q, b.start, b.length, b.table, out, scale=float("nan")) == L.LSCD_ERROR_INVALID_VALUE
    assert status(b.handle, c, b.q, b.start, b.length, b.table, out, window=-1) == L.LSCD_ERROR_INVALID_VALUE
    other = L.lscd_attention_create(4, 4, 64)
    assert status(other, c, b.q, b.start, b.length, b.table, out) == L.LSCD_ERROR_INVALID_VALUE
    for args, want in (((3, 2, 64), L.LSCD_ERROR_INVALID_VALUE), ((4, 2, 40), L.LSCD_ERROR_NOT_SUPPORTED),
                       ((4, 2, 272), L.LSCD_ERROR_NOT_SUPPORTED), ((0, 1, 64), L.LSCD_ERROR_INVALID_VALUE)):
        with pytest.raises(L.LSCDError) as e:
            L.lscd_attention_create(*args)
        assert e.value.status == want
