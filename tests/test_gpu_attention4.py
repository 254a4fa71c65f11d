"""Attention over a paged cache of 4-bit codes, and the logarithms of the rows' sums over every kind of cache,
on the GPU against the plain 64-bit definition.

Outputs: the tolerance of test_gpu_attention (the codes' values are exact in both 16-bit types here).
Logarithms: s_j = scale q.k_j is off by at most d = (dim + 8) 2^-24 of sum |scale q k| (products of 16-bit values
are exact, dim sums and the scaling round), so is ln sum exp(s_j); 2^-20 for exponentials and the logarithm;
(length / 16 + 64) 2^-24 for sums in sequence (a lane has one position in 16, then come the joins);
2^-22 of the result and of sum |scale q k| for its units (log2, ln) and the subtraction of the maximum.
"""
import numpy as np
import pytest

from oracle import serving as sv
from tests._util import say
from tests.test_gpu_attention import CHUNKS, DECODE, Batch
from tests.test_gpu_attention_edges import place

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L


class Batch4(Batch):
    """The same over random 4-bit codes with scales 2^-2 and 2^-1; bytes that belong to nobody are 255."""

    def __init__(self, seqs, heads, kv, dim, page, kind, cache="e2m1", seed=0, **more):
        super().__init__(seqs, heads, kv, dim, page, kind, kind if cache == "e2m1" else cache, seed=seed, **more)
        if cache != "e2m1":
            return
        g = torch.Generator().manual_seed(seed + 1)
        shape, row = (self.pages, kv, page), 2 if dim <= 64 else 4 if dim <= 128 else 8
        codes = [torch.randint(0, 256, shape + (dim // 2,), generator=g, dtype=torch.uint8) for _ in range(2)]
        scales = [torch.randint(125, 127, shape + (row,), generator=g, dtype=torch.uint8) for _ in range(2)]
        for x in scales:
            x[..., (dim + 31) // 32:] = 255
        self.tensors = [x.cuda() for x in codes + scales]

    def values(self, which, i):
        if self.tensors[which].dtype != torch.uint8:
            return super().values(which, i)
        x = sv.e2m1_values(self.tensors[which].cpu().numpy(), self.tensors[2 + which].cpu().numpy(), self.dim)
        n = self.seqs[i][1]
        pages = self.table[i, :(n + self.page - 1) // self.page].long().cpu().numpy()
        return x[pages].transpose(0, 2, 1, 3).reshape(-1, self.kv, self.dim)[:n]

    def run_lse(self, **kw):
        lse = torch.full((self.T, self.heads), 123.0, device="cuda")
        return self.run(lse=lse, **kw), lse

    def check_lse(self, lse, scale=None, causal=True, window=0):
        scale = self.dim ** -0.5 if scale is None else scale
        at, got, q = 0, lse.cpu().double().numpy(), self.q.cpu().double().numpy()
        for i, (n, length) in enumerate(self.seqs):
            k = self.values(0, i)
            for t in range(n):
                p = length - n + t
                j = np.arange(length)
                seen = (j <= p if causal else j >= 0) & ((j > p - window) if window else True)
                for h in range(self.heads):
                    s = scale * (k[seen, h // (self.heads // self.kv)] @ q[at + t, h])
                    if not seen.any():
                        assert got[at + t, h] == -np.inf
                        continue
                    want = s.max() + np.log(np.exp(s - s.max()).sum())
                    big = (np.abs(scale * k[seen, h // (self.heads // self.kv)]) @ np.abs(q[at + t, h])).max()
                    tol = (self.dim + 8) * 2.0 ** -24 * big + 2.0 ** -20 + (length / 16 + 64) * 2.0 ** -24 + 2.0 ** -22 * (abs(want) + big)
                    assert abs(got[at + t, h] - want) <= tol, (i, t, h, got[at + t, h], want, tol)
            at += n


SHAPES = [(2, 2, 128, 16), (8, 2, 128, 32), (16, 1, 64, 64), (3, 3, 80, 16), (20, 1, 256, 16), (4, 4, 16, 128), (2, 2, 48, 16),
          (2, 1, 112, 16), (2, 2, 144, 32), (4, 2, 240, 16)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,dim,page", SHAPES)
def test_decode(heads, kv, dim, page, kind):
    say(f"decode {heads}/{kv} x {dim}, page {page}, {kind} over e2m1")
    b = Batch4(DECODE, heads, kv, dim, page, kind, seed=dim + heads)
    out, lse = b.run_lse()
    assert torch.equal(out, b.run())
    b.check(out)
    b.check_lse(lse)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,dim,page", [(2, 2, 128, 16), (4, 1, 128, 64), (6, 2, 64, 16), (2, 2, 80, 32), (2, 1, 256, 16),
                                               (2, 2, 112, 16), (2, 2, 160, 16), (2, 2, 16, 16)])
def test_chunks(heads, kv, dim, page, kind):
    say(f"chunks {heads}/{kv} x {dim}, page {page}, {kind} over e2m1")
    b = Batch4(CHUNKS, heads, kv, dim, page, kind, seed=dim + heads)
    out, lse = b.run_lse()
    assert torch.equal(out, b.run())
    b.check(out)
    b.check_lse(lse)


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "bf16"), ("f16", "e4m3"), ("bf16", "e4m3")])
@pytest.mark.parametrize("seqs", [DECODE, [(130, 130), (64, 300), (0, 0), (1, 77), (5, 40)], [(40, 1500)]])
@pytest.mark.parametrize("dim", [64, 128, 256])
def test_logarithms_over_other_caches(seqs, kind, cache, dim):
    say("lse", seqs, kind, cache, dim)
    b = Batch4(seqs, 4, 2, dim, 16, kind, cache, seed=dim)
    out, lse = b.run_lse()
    assert torch.equal(out, b.run())
    b.check_lse(lse)


@pytest.mark.parametrize("seqs", [[(1, 900), (1, 50), (1, 300)], [(3, 700), (2, 40)], [(200, 600), (7, 300), (1, 299)],
                                  [(4, 2), (1, 0), (3, 3)], [(200, 90), (100, 0), (5, 1)]])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 33), (False, 0), (False, 100)])
def test_masks(seqs, causal, window):
    """Windows, no causality, rows that see nothing."""
    say("masks", seqs, causal, window)
    b = Batch4(seqs, 4, 2, 64, 16, "f16", seed=window)
    out, lse = b.run_lse(causal=causal, window=window)
    b.check(out, causal=causal, window=window)
    b.check_lse(lse, causal=causal, window=window)


@pytest.mark.parametrize("scale", [0.0, -0.2, 3000.0])
def test_scale(scale):
    say("scale", scale)
    b = Batch4([(1, 300), (40, 200)], 4, 4, 64, 16, "f16", seed=4)
    out, lse = b.run_lse(scale=scale)
    if scale < 3000:  # (there scores of 2^-24 of thousands decide; their logarithms' tolerance says so)
        b.check(out, scale=scale)
    b.check_lse(lse, scale=scale)


def test_a_long_sequence_among_short_ones():
    """Parts of both kernels joined: 39 and more of few rows, cut items of many."""
    say("long and short")
    for seqs, share in (([(1, 9000)] + [(1, 1 + 37 * i % 200) for i in range(20)], 2), ([(2, 20000)], 1), ([(60, 6000), (1, 50), (20, 40)], 2)):
        b = Batch4(seqs, 2 * share, 2, 64, 16, "f16", seed=1)
        out, lse = b.run_lse()
        b.check(out)
        b.check_lse(lse)
        for _ in range(3):
            again = b.run_lse()
            assert torch.equal(again[0], out) and torch.equal(again[1], lse)


@pytest.mark.parametrize("n,heads", [(4, 4), (100, 2), (7, 2), (1, 2)])
@pytest.mark.parametrize("dim", [64, 80, 128])
def test_groups_that_are_not_numbers(n, heads, dim):
    """A scale byte of 255 in new token j reaches tokens j.. only, and of the values its own 32 channels only; none
    before a window, behind the last position or in a page of no sequence reaches anybody."""
    say("groups of NaN", n, heads, dim)
    length, page = 150, 16
    b = Batch4([(n, length)], heads, 2, dim, page, "f16", seed=n)
    clean = b.run()
    j = n // 2
    at = length - n + j
    slot = (b.table[0, at // page].long(), slice(None), at % page)
    for which in (2, 3):
        keep = b.tensors[which][slot].clone()
        b.tensors[which][slot[0], :, slot[2], 1] = 255
        out, lse = b.run_lse()
        assert torch.equal(out[:j], clean[:j]), which
        if which == 3:
            assert not torch.isfinite(out[j:, :, 32:64]).any()
            assert torch.equal(out[j:, :, :32], clean[j:, :, :32]) and torch.equal(out[j:, :, 64:], clean[j:, :, 64:])
            b.check_lse(lse)
        windowed = b.run(window=1)                           # token i sees position at - j + i only
        assert torch.isfinite(windowed[torch.arange(n) != j]).all()
        b.tensors[which][slot] = keep
    seen = b.run(window=40)
    used = torch.zeros((b.pages, page), dtype=torch.bool)
    for j in range(max(0, length - n - 39), length):
        used[b.table[0, j // page].long(), j % page] = True
    for which in (2, 3):
        b.tensors[which].masked_fill_(~used[:, None, :, None].cuda(), 255)
    assert torch.equal(b.run(window=40), seen)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 40])
def test_values_past_the_largest_count_as_the_largest(kind, n):
    """Codes that stand for more than the type holds, among the keys (times zero in the query) and the values."""
    say("largest values", kind, n)
    length, dim = 70, 128
    b = Batch4([(n, length)], 2, 2, dim, 16, kind, seed=5)
    top = 14 if kind == "f16" else 126
    largest = 65504.0
    b.q[:, :, 32:64] = 0
    for j in range(length):
        place(b, 2, 0, j, torch.tensor([126, 127 + top, 126, 126], dtype=torch.uint8, device="cuda"))
        place(b, 0, 0, j, torch.full((dim // 2,), 0x77, dtype=torch.uint8, device="cuda"))
        place(b, 3, 0, j, torch.tensor([126, 126, 127 + top, 126], dtype=torch.uint8, device="cuda"))
        place(b, 1, 0, j, torch.tensor([0x22] * 32 + [0x77] * 16 + [0x22] * 16, dtype=torch.uint8, device="cuda"))
    out = b.run()                                            # equal keys: a mean of equal values
    want = torch.full((dim,), 0.5, dtype=torch.float64)
    # (sums are fp32 and taken before the division by the weights' sum: two of bfloat16's largest, 2 * 3.39e38, pass
    # fp32's largest, 3.40e38; 70 times 65504 with weights of up to 2^15 stay far below it)
    want[64:96] = largest if kind == "f16" else np.inf
    assert torch.equal(out.cpu().double(), want.expand(n, 2, dim))


def test_prefix_and_rest_joined():
    """Outputs over two parts of a cache, weighed by their logarithms, are the output over the whole."""
    say("joined")
    b = Batch4([(1, 200)], 4, 2, 64, 16, "f16", seed=7)
    whole, lse = b.run_lse()
    parts = []
    for table, n in ((b.table[:, :5], 80), (b.table[:, 5:], 120)):
        o, s = torch.empty_like(whole), torch.empty_like(lse)
        L.lscd_attention(b.handle, b.cache(), b.q, b.start, torch.full_like(b.length, n), table, o, causal=False, lse=s)
        parts.append((o.double(), s.double()))
    w = torch.softmax(torch.stack([s for _, s in parts]), 0)
    got = sum(o * x[..., None] for (o, _), x in zip(parts, w))
    # three roundings to float16 of numbers up to max |v|, and of the weights in each
    top = max(float(o.abs().max()) for o, _ in parts)
    assert float((got - whole.double()).abs().max()) <= 4 * 2.0 ** -11 * top
    assert float((torch.logsumexp(torch.stack([s for _, s in parts]), 0) - lse.double()).abs().max()) <= 1e-5


def test_rows_behind_the_last_sequence_stay():
    say("rows behind")
    b = Batch4([(1, 60), (20, 90)], 4, 2, 64, 16, "f16", seed=6)
    for share_start in ([0, 1, 21], [0, 1, 9]):
        b.start.copy_(torch.tensor(share_start, dtype=torch.int32))
        out = torch.full_like(b.q, 3.0)
        lse = torch.full((b.T, 4), 3.0, device="cuda")
        b.run(out=out, lse=lse)
        assert (out[share_start[-1]:] == 3).all() and (lse[share_start[-1]:] == 3).all()
        assert not (lse[:share_start[-1]] == 3).any()


def test_offsets_past_32_bits():
    """Pages at the end of a pool of more than 2^31 bytes."""
    say("large pool")
    b = Batch4([(1, 100), (30, 90)], 8, 8, 128, 16, "f16", seed=12)
    pages = (2 ** 31 + 2 ** 27) // (8 * 16 * 64)
    big = [torch.empty((pages, *x.shape[1:]), dtype=torch.uint8, device="cuda") for x in b.tensors]
    for x, y in zip(big, b.tensors):
        x[pages - b.pages:] = y
    small = b.run()
    b.check(small)
    b.tensors, b.table = big, torch.where(b.table < 0, b.table, b.table + (pages - b.pages)).to(torch.int32)
    assert torch.equal(b.run(), small)


def test_contents_out_of_range_are_clamped():
    say("clamped contents")
    for n in (1, 50):
        b = Batch4([(n, 60), (n, 30)], 4, 2, 64, 16, "f16", seed=3)
        b.length[0] = 2 ** 30
        b.table[1, 0] = 2 ** 30
        b.start[2] = 2 ** 30
        out, _ = b.run_lse()
        assert out.shape[0] == 2 * n


def test_stream_and_graph():
    say("stream, graph")
    for seqs in ([(1, 300), (1, 20)], [(40, 300), (1, 20), (3, 64)]):
        b = Batch4(seqs, 4, 2, 64, 16, "f16", seed=11)
        want, log = b.run_lse()
        out, lse, cache = torch.empty_like(want), torch.empty_like(log), b.cache()
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            L.lscd_attention(b.handle, cache, b.q, b.start, b.length, b.table, out, lse=lse)
        s.synchronize()
        assert torch.equal(out, want) and torch.equal(lse, log)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lscd_attention(b.handle, cache, b.q, b.start, b.length, b.table, out, lse=lse)
        for k in range(4):
            b.length.copy_(torch.tensor([n - 3 * k for _, n in seqs], dtype=torch.int32))
            b.q.normal_()
            graph.replay()
            torch.cuda.synchronize()
            eager = b.run_lse()
            assert torch.equal(out, eager[0]) and torch.equal(lse, eager[1])


def test_refusals():
    say("refusals")
    b = Batch4([(1, 60), (20, 90)], 4, 2, 64, 16, "f16")
    out = torch.empty_like(b.q)
    good = torch.empty((b.T, 4), device="cuda")
    for bad in (good.half(), good[:-1], good[:, :2], torch.empty((4, b.T), device="cuda").t(), good.cpu()):
        with pytest.raises(ValueError):
            L.lscd_attention(b.handle, b.cache(), b.q, b.start, b.length, b.table, out, lse=bad)
    args = (b.handle.ptr, b.cache().ptr, b.q.data_ptr(), 256, b.start.data_ptr(), b.length.data_ptr(), b.table.data_ptr(),
            b.table.shape[1], b.table.shape[1], 2, b.T, 0.125, 1, 0, out.data_ptr(), 256)
    assert L._lib.lscd_attention_lse(*args, None, L.LSCD_F16, None) == L.LSCD_ERROR_INVALID_VALUE
    assert L._lib.lscd_attention_lse(*args, good.data_ptr() + 2, L.LSCD_F16, None) == L.LSCD_ERROR_INVALID_VALUE
