"""Eviction from a paged cache (lscd_cache_evict) on the GPU, bit for bit against the definition: the positions
that are kept, the keys, values, scales and weights that move, and everything else as it was."""
import numpy as np
import pytest

from tests._util import say

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L

BYTES = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.uint8, "e2m1": torch.uint8}


class Pool:
    """Random bytes in every row, random weights, shuffled pages for sequences of the given lengths and for `to`."""

    def __init__(self, lengths, keep, heads, dim, page, kind, seed=0, spare=3):
        g = torch.Generator().manual_seed(seed)
        self.lengths, self.keep, self.heads, self.dim, self.page, self.kind = lengths, keep, heads, dim, page, kind
        need = [(n + page - 1) // page for n in lengths]
        self.wide, self.to_wide = max(need + [1]) + 1, (keep + page - 1) // page
        self.pages = sum(need) + len(lengths) * self.to_wide + spare
        shape = (self.pages, heads, page)
        row = {"f16": 2 * dim, "bf16": 2 * dim, "e4m3": dim, "e2m1": dim // 2}[kind]
        scale = {"e4m3": 4, "e2m1": 2 if dim <= 64 else 4 if dim <= 128 else 8}.get(kind, 0)
        self.raw = [torch.randint(0, 256, shape + (n,), generator=g, dtype=torch.uint8) for n in (row, row, scale, scale)]
        self.weight = torch.rand(shape, generator=g) ** 8
        order, at = torch.randperm(self.pages, generator=g).to(torch.int32), 0
        self.table = torch.full((len(lengths), self.wide), -1, dtype=torch.int32)
        self.to = torch.full((len(lengths), self.to_wide + 2), -1, dtype=torch.int32)
        for i, n in enumerate(need):
            self.table[i, :n] = order[at:at + n]
            at += n
            self.to[i, :self.to_wide] = order[at:at + self.to_wide]
            at += self.to_wide
        self.device()

    def device(self):
        """Fresh copies on the GPU."""
        x = [t.cuda() for t in self.raw]
        if self.kind == "e2m1":
            self.tensors = x
        elif self.kind == "e4m3":
            self.tensors = [x[0].view(torch.float8_e4m3fn), x[1].view(torch.float8_e4m3fn)] + \
                [t.view(torch.float32).squeeze(-1) for t in x[2:]]
        else:
            self.tensors = [t.view(BYTES[self.kind]) for t in x[:2]]
        self.bytes, self.w = x, self.weight.cuda()
        self.args = [torch.tensor(self.lengths, dtype=torch.int32).cuda(), self.table.cuda()]
        return L.Cache(*self.tensors)

    def expect(self, recent, to):
        """(kept, raw, weight) by the definition, one sequence and head at a time."""
        kept = np.full((len(self.lengths), self.heads, self.keep), -1, dtype=np.int32)
        raw, weight = [t.numpy().copy() for t in self.raw], self.weight.numpy().copy()
        dest = self.to if to else self.table
        for s, n in enumerate(self.lengths):
            if n == 0:
                continue
            last = min(recent, min(n, self.keep))
            pos = np.arange(n)
            p, r = self.table[s, :self.wide].numpy()[pos // self.page], pos % self.page
            for h in range(self.heads):
                w = self.weight.numpy()[p, h, r].astype(np.float64)
                w = np.where(np.isnan(w), np.inf, w)          # (no infinities among the weights of the tests with NaN)
                best = sorted(range(n - last), key=lambda j: (-w[j], j))[:min(n, self.keep) - last]
                mine = np.array(sorted(best) + list(range(n - last, n)), dtype=np.int64)
                kept[s, h, :len(mine)] = mine
                if not to and n <= self.keep:
                    continue
                i = np.arange(len(mine))
                q = dest[s].numpy()[i // self.page]
                for x, y in zip(self.raw + [self.weight], raw + [weight]):
                    y[q, h, i % self.page] = x.numpy()[p[mine], h, r[mine]]
        return kept, raw, weight

    def check(self, recent=0, to=False):
        cache = self.device()
        kept = L.lscd_cache_evict(cache, self.w, *self.args, self.keep, recent, to=self.to.cuda() if to else None)
        torch.cuda.synchronize()
        want = self.expect(recent, to)
        assert np.array_equal(kept.cpu().numpy(), want[0])
        for x, y in zip(self.bytes, want[1]):
            assert np.array_equal(x.cpu().numpy(), y)
        assert np.array_equal(self.w.cpu().numpy().view(np.int32), want[2].view(np.int32))


@pytest.mark.parametrize("kind", ["f16", "e4m3", "e2m1"])
@pytest.mark.parametrize("heads,dim,page", [(1, 16, 16), (3, 64, 16), (2, 80, 32), (2, 128, 64), (1, 256, 16), (2, 48, 128), (1, 240, 16)])
@pytest.mark.parametrize("to", [False, True])
def test_rows(heads, dim, page, kind, to):
    """All row sizes; sequences shorter than, equal to and longer than what is kept."""
    say("rows", heads, dim, page, kind, to)
    Pool([200, 0, 1, 63, 64, 65, 150], 64, heads, dim, page, kind, seed=dim + heads).check(20, to)


@pytest.mark.parametrize("keep,recent", [(1, 0), (1, 1), (16, 16), (17, 3), (300, 0), (300, 100), (299, 298), (1024, 7)])
@pytest.mark.parametrize("to", [False, True])
def test_how_many(keep, recent, to):
    say("keep", keep, recent, to)
    Pool([1500, 299, 300, 301, 17, 1025], keep, 2, 64, 16, "e4m3", seed=keep).check(recent, to)


@pytest.mark.parametrize("n,keep", [(16384, 5000), (16385, 1000), (36864, 20000), (37001, 2000), (70000, 30000)])
@pytest.mark.parametrize("to", [False, True])
def test_long_sequences(n, keep, to):
    """Weights that LDS holds and that it does not; many rounds of rows in place."""
    say("long", n, keep, to)
    Pool([n, n // 3], keep, 2, 16, 64, "f16", seed=n).check(100, to)


@pytest.mark.parametrize("to", [False, True])
def test_weights_of_all_kinds(to):
    """Equal weights keep the lower position; zeros of both signs are equal; negative ones, subnormals, NaN."""
    say("kinds of weights", to)
    for seed in range(6):
        p = Pool([500, 130, 40], 48, 3, 16, 16, "f16", seed=seed)
        g = torch.Generator().manual_seed(seed)
        few = torch.tensor([[0.0, -0.0, 1.0], [0.25, 0.25, 0.25], [-1.0, -2.0, -0.0], [1e-40, 2e-40, 0.0],
                            [float("nan"), 1.0, -float("nan")], [3e38, -3e38, 0.5]][seed])
        p.weight = few[torch.randint(0, 3, p.weight.shape, generator=g)]
        p.check(5, to)


def test_one_bit_of_difference():
    """Weights that differ in the last bits only, whose first digits are all equal."""
    say("last bits")
    p = Pool([3000], 700, 2, 16, 16, "f16", seed=3)
    g = torch.Generator().manual_seed(9)
    p.weight = (0x3F000000 + torch.randint(0, 2000, p.weight.shape, generator=g)).to(torch.int32).view(torch.float32)
    p.check(0, True)
    p.check(0, False)


def test_after_the_weights():
    """What the attention over the rest sees: with `keep` of all positions it sees what it saw; later tokens go behind."""
    say("weigh, evict, attend")
    heads, kv, dim, page, n, keep = 4, 2, 64, 16, 400, 100
    g = torch.Generator().manual_seed(2)
    pages = 40
    cache = L.Cache(*(torch.randint(0, 256, (pages, kv, page, dim // 2), generator=g, dtype=torch.uint8).cuda() for _ in range(2)),
                    *(torch.full((pages, kv, page, 2), 125, dtype=torch.uint8).cuda() for _ in range(2)))
    weight = torch.full((pages, kv, page), 77.0, device="cuda")
    table = torch.randperm(pages, generator=g)[None, :n // page].to(torch.int32).cuda()
    q = torch.randn((n, heads, dim), generator=g).half().cuda()
    o, lse = torch.empty_like(q), torch.empty((n, heads), device="cuda")
    att = L.lscd_attention_create(heads, kv, dim)
    ints = lambda *v: torch.tensor(v, dtype=torch.int32, device="cuda")  # noqa: E731
    L.lscd_attention(att, cache, q, ints(0, n), ints(n), table, o, lse=lse)
    L.lscd_cache_weigh(cache, q, lse, ints(0, n), ints(n), table, weight)
    slots = (table[0].long()[torch.arange(n, device="cuda") // page] * page + torch.arange(n, device="cuda") % page).to(torch.int32)
    k, v = (torch.empty((n, kv, dim), dtype=torch.float16, device="cuda") for _ in range(2))
    L.lscd_cache_read(cache, slots, k, v)
    w = weight[table[0].long()].permute(1, 0, 2).reshape(kv, n).clone()
    kept = L.lscd_cache_evict(cache, weight, ints(n), table, keep, 16)
    for h in range(kv):
        best = torch.sort(torch.sort(w[h, :n - 16], descending=True, stable=True)[1][:keep - 16])[0]
        assert torch.equal(kept[0, h].long(), torch.cat([best, torch.arange(n - 16, n, device="cuda")]))
    k2, v2 = (torch.empty((keep, kv, dim), dtype=torch.float16, device="cuda") for _ in range(2))
    L.lscd_cache_read(cache, slots[:keep], k2, v2)
    for h in range(kv):
        assert torch.equal(k2[:, h], k[kept[0, h].long(), h]) and torch.equal(v2[:, h], v[kept[0, h].long(), h])
        assert torch.equal(weight[table[0].long()].permute(1, 0, 2).reshape(kv, n)[h, :keep], w[h, kept[0, h].long()])
    # one more token behind what is left
    L.lscd_cache_write(cache, k[:1] * 0.5, v[:1], slots[keep:keep + 1])
    L.lscd_attention(att, cache, q[:1], ints(0, 1), ints(keep + 1), table, o[:1], lse=lse[:1])
    L.lscd_cache_weigh(cache, q[:1], lse[:1], ints(0, 1), ints(keep + 1), table, weight)
    L.lscd_cache_read(cache, slots[:keep + 1], *(x := [torch.empty((keep + 1, kv, dim), dtype=torch.float16, device="cuda") for _ in range(2)]))
    for f in range(heads):
        p = torch.softmax(q[0, f].double() @ x[0][:, f // 2].double().t() * dim ** -0.5, 0)
        want = p @ x[1][:, f // 2].double()
        # (the output's and the weights' rounding, 2^-11 each, of values up to max |v|)
        assert float((o[0, f].double() - want).abs().max()) <= 2 * 2.0 ** -11 * float(x[1].abs().max())


def test_offsets_past_32_bits():
    """Rows and weights at the end of a pool of more than 2^32 bytes."""
    say("large pool")
    p = Pool([300, 40], 64, 8, 128, 16, "f16", seed=12)
    pages = (2 ** 31 + 2 ** 27) // (8 * 16 * 128)
    at = pages - p.pages
    want = p.expect(10, False)
    big = [torch.zeros((pages, 8, 16, 128), dtype=torch.float16, device="cuda") for _ in range(2)]
    for x, y in zip(big, p.tensors):
        x[at:] = y
    weight = torch.zeros((pages, 8, 16), device="cuda")
    weight[at:] = p.w
    table = torch.where(p.table < 0, p.table, p.table + at).to(torch.int32).cuda()
    kept = L.lscd_cache_evict(L.Cache(*big), weight, p.args[0], table, 64, 10)
    assert np.array_equal(kept.cpu().numpy(), want[0])
    for x, y in zip(big, want[1]):
        assert np.array_equal(x[at:].view(torch.uint8).cpu().numpy(), y) and not x[:at].any()
    assert np.array_equal(weight[at:].cpu().numpy(), want[2])


def test_contents_out_of_range_are_clamped():
    """Lengths past the table or negative, pages outside the pool, in either table: no access out of bounds."""
    say("clamped contents")
    for to in (False, True):
        p = Pool([200, 100, 50], 32, 2, 64, 16, "e4m3", seed=4)
        cache = p.device()
        p.args[0].copy_(torch.tensor([2 ** 30, -5, 2 ** 30], dtype=torch.int32))
        p.args[1][0, 2] = 2 ** 30
        dest = p.to.cuda()
        dest[2, 1] = -7
        kept = L.lscd_cache_evict(cache, p.w, *p.args, 32, 8, to=dest if to else None).cpu()
        assert (kept[1] == -1).all() and (kept[0] >= 0).all() and (kept < p.wide * 16).all()
        assert (kept[0, :, 1:] > kept[0, :, :-1]).all()


def test_strides_stream_and_graph():
    say("strides, stream, graph")
    p = Pool([300, 90, 500], 64, 2, 80, 16, "e2m1", seed=6)
    want = p.expect(9, True)
    cache = p.device()
    tables = [torch.full((3, t.shape[1] + 5), 9, dtype=torch.int32, device="cuda") for t in (p.table, p.to)]
    for x, t in zip(tables, (p.table, p.to)):
        x[:, :t.shape[1]] = t
    table, to = (x[:, :t.shape[1]] for x, t in zip(tables, (p.table, p.to)))
    kept = torch.empty((3, 2, 64), dtype=torch.int32, device="cuda")
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.lscd_cache_evict(cache, p.w, p.args[0], table, 64, 9, to=to, kept=kept)
    s.synchronize()
    assert np.array_equal(kept.cpu().numpy(), want[0]) and np.array_equal(p.bytes[1].cpu().numpy(), want[1][1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lscd_cache_evict(cache, p.w, p.args[0], table, 64, 9, kept=kept)
    for lengths in ([300, 90, 500], [100, 64, 65], [500, 0, 77]):
        p.lengths = [min(n, (p.table[i] >= 0).sum().item() * 16) for i, n in enumerate(lengths)]
        want = p.expect(9, False)
        for x, y in zip(p.bytes, p.raw):
            x.copy_(y)
        p.w.copy_(p.weight)
        p.args[0].copy_(torch.tensor(p.lengths, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        assert np.array_equal(kept.cpu().numpy(), want[0])
        assert all(np.array_equal(x.cpu().numpy(), y) for x, y in zip(p.bytes, want[1]))
        assert np.array_equal(p.w.cpu().numpy(), want[2])


def test_nothing_to_do_and_refusals():
    say("refusals")
    p = Pool([100, 40], 32, 2, 64, 16, "f16", seed=1)
    c = p.device()
    assert L.lscd_cache_evict(c, p.w, p.args[0][:0], p.args[1][:0], 32).shape == (0, 2, 32)

    def status(*args, **kw):
        with pytest.raises(L.LSCDError) as e:
            L.lscd_cache_evict(c, p.w, *p.args, *args, **kw)
        return e.value.status

    for args, kw in (((0,), {}), ((32, -1), {}), ((32, 33), {}), ((32, 0), dict(to=p.to.cuda()[:, :1]))):
        assert status(*args, **kw) == L.LSCD_ERROR_INVALID_VALUE
    for weight, length, table, kw in (
            (p.w[:-1], *p.args, {}), (p.w.half(), *p.args, {}), (p.w, p.args[0].long(), p.args[1], {}),
            (p.w, p.args[0], p.args[1][:1], {}), (p.w, *p.args, dict(to=p.to.cuda()[:1])),
            (p.w, *p.args, dict(kept=torch.empty((2, 2, 31), dtype=torch.int32, device="cuda"))),
            (p.w, *p.args, dict(kept=torch.empty((2, 2, 32), dtype=torch.int64, device="cuda")))):
        with pytest.raises(ValueError):
            L.lscd_cache_evict(c, weight, length, table, 32, **kw)
    assert all(torch.equal(x.cpu(), y) for x, y in zip(p.bytes, p.raw)) and torch.equal(p.w.cpu(), p.weight)


def test_twice_in_place_is_once():
    """A sequence that has been cut stays as it is when the call is made again with its new length."""
    say("twice")
    p = Pool([400, 90], 64, 2, 64, 16, "e4m3", seed=8)
    cache = p.device()
    L.lscd_cache_evict(cache, p.w, *p.args, 64, 10)
    p.args[0].clamp_(max=64)
    before, w = [x.clone() for x in p.bytes], p.w.clone()
    kept = L.lscd_cache_evict(cache, p.w, *p.args, 64, 10)
    assert torch.equal(kept, torch.arange(64, device="cuda", dtype=torch.int32).expand(2, 2, 64))
    assert all(torch.equal(x, y) for x, y in zip(before, p.bytes)) and torch.equal(p.w, w)
