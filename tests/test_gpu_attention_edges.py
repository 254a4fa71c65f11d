"""Attention over a paged cache at the ends of its types' ranges and of its arguments.

Tolerances are those of test_gpu_attention (u: unit roundoff, A = sum_j p_j |v_j|), with the floor of small
float16 weights written out: a weight is rounded to a step of at most 2^-31 of the largest, so to within
2^-32 of it, which is 2^-32 / sum_j exp(s_j - max s) of the whole.
"""
import numpy as np
import pytest

from oracle import serving as sv
from tests._util import say
from tests.test_gpu_attention import TYPES, Batch

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L


def place(b, which, i, j, value):
    """Set position j of sequence i (all heads)."""
    b.tensors[which][b.table[i, j // b.page].long(), :, j % b.page] = value


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("d", [9.5, 12.0, 16.0, 17.5, 20.0])
def test_weights_far_below_the_largest(kind, n, d):
    """One position in 32 holds a large score and nothing else; the rest, d nats lower, hold what is there to sum."""
    say("small weights", kind, n, d)
    length = 1000
    b = Batch([(n, length)], 2, 2, 64, 16, kind, kind)
    b.q.zero_()
    b.q[:, :, 0] = 1
    for x, rest in zip(b.tensors, (-d, 1024.0)):
        x.zero_()
        for j in range(length):
            if j % 32:
                place(b, 0 if rest < 0 else 1, 0, j, torch.tensor([rest] + [0.0] * 63 if rest < 0 else [rest] * 64).to(x))
    got = b.run(scale=1.0).cpu().double().numpy()
    o, a, big = sv.attention(b.q.cpu().double().numpy(), b.values(0, 0), b.values(1, 0), 1.0)
    u, e = sv.ROUNDOFF[kind], 2 * (64 + 8) * 2.0 ** -24 * big[..., None] + 2.0 ** -18
    tol = u * np.abs(o) + (u + e) * a + sv.TINY[kind]
    for i in range(n):
        seen = np.arange(length - n + i + 1) % 32 != 0
        total = (~seen).sum() + seen.sum() * np.exp(-d)
        tol[i] += (2.0 ** -32 if kind == "f16" else 0.0) * seen.sum() * 1024 / total
    assert (np.abs(got - o) <= tol).all(), float((np.abs(got - o) / tol).max())


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("seqs", [[(1, 3), (1, 20), (1, 300), (5, 40)], [(100, 230)]])
def test_equal_values_come_out_as_they_are(seqs, kind):
    """The weights that are summed are those that are multiplied: a mean of equal values is that value."""
    say("equal values", seqs, kind)
    b = Batch(seqs, 4, 2, 64, 16, kind, kind, seed=9)
    b.tensors[1].copy_(torch.linspace(1, 2, 64).to(b.tensors[1]))
    assert torch.equal(b.run(), torch.linspace(1, 2, 64).to(b.q).expand(b.q.shape))


@pytest.mark.parametrize("kind,scale", [("f16", 2.0 ** 22), ("f16", 2.0 ** 32), ("bf16", 2.0 ** 22), ("bf16", 2.0 ** 60), ("bf16", 2.0 ** 110)])
@pytest.mark.parametrize("n", [1, 40])
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_of_any_size(kind, scale, n, sign):
    """Scores far beyond the exponential's range, up to fp32's: equal ones weigh the same, smaller ones nothing.

    Keys are equal but for one position in seven, whose score is far lower: what is left is a mean of the other
    values, whose weights are equal (error: the output's rounding, and 2^-18 for the sums)."""
    say("scores of any size", kind, scale, n, sign)
    length, half = 150, scale ** 0.5
    b = Batch([(n, length)], 2, 2, 64, 16, kind, kind, seed=3)
    b.q.zero_()
    b.q[:, :, :3] = torch.tensor([1.0, 1.0, 0.5]).to(b.q) * 1.1 * sign * (half if kind == "bf16" else 2.0 ** 8)
    k = torch.tensor([1.0, 0.75, 1.0] + [0.0] * 61) * 1.3 * (half if kind == "bf16" else 2.0 ** 8)
    for j in range(length):
        place(b, 0, 0, j, (k * (0.5 if (j % 7 == 3) == (sign > 0) else 1.0)).to(b.q))
    got = b.run(scale=0.3 if kind == "bf16" else 0.3 * scale / 2 ** 16).cpu().double().numpy()
    v = b.values(1, 0)
    for i in range(n):
        j = np.arange(length - n + i + 1)
        best = v[j[j % 7 != 3]]
        want, a = best.mean(0), np.abs(best).mean(0)
        assert (np.abs(got[i] - want) <= sv.ROUNDOFF[kind] * np.abs(want) + 2.0 ** -18 * a + sv.TINY[kind]).all(), i


@pytest.mark.parametrize("seqs", [[(5, 40)], [(5, 40), (0, 90)], [(1, 40)], [(30, 70), (2, 9)], [(0, 12)]])
def test_fewer_tokens_than_rows(seqs):
    """Room for 64 tokens and starts that end before: those tokens are served, the other rows stay."""
    say("fewer tokens than rows", seqs)
    b = Batch(seqs, 4, 2, 64, 16, "f16", "f16", seed=21)
    used, spare = b.T, 64 - b.T
    q = torch.cat([b.q, torch.full((spare, 4, 64), float("nan"), dtype=torch.float16, device="cuda")])
    out = b.run(q=q, out=torch.full_like(q, 7.0))
    b.check(out[:used])
    assert (out[used:] == 7).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("n,length", [(1, 64), (2, 50), (40, 64), (40, 200)])
def test_codes_past_the_largest_value(kind, n, length):
    """The largest 16-bit values are stored as codes that stand for a little more (65536 for 65504): they count as the
    type's largest value, one unit roundoff less (u A, and in the scores what q makes of the difference)."""
    say("codes past the largest value", kind, n, length)
    b = Batch([(n, length)], 2, 2, 64, 16, kind, "e4m3", seed=14)
    top = float(torch.finfo(TYPES[kind]).max)
    k, v = (torch.randn((length, 2, 64), device="cuda").to(TYPES[kind]) for _ in range(2))
    k[7, :, 3], k[9, :, 5], v[5, :, 1], v[5, :, 2] = top, -top, top, -top
    b.q[:, :, 3] = 0.0
    b.q[:, :, 5] = 2.0 / top
    place = torch.arange(length, device="cuda")
    slots = (b.table[0, place // 16] * 16 + place % 16).to(torch.int32)
    L.lscd_cache_write(b.cache(), k, v, slots)
    got = b.run().cpu().double().numpy()
    assert np.abs(b.values(1, 0)).max() > top
    o, a, big = sv.attention(b.q.cpu().double().numpy(), b.values(0, 0), b.values(1, 0), 64 ** -0.5)
    u = sv.ROUNDOFF[kind]
    e = 2 * (64 + 8) * 2.0 ** -24 * big[..., None] + 2 * 64 ** -0.5 * 2 * u + 2.0 ** -18
    assert (np.abs(got - o) <= u * np.abs(o) + (2 * u + e) * a + sv.TINY[kind]).all()


def test_wide_tables_are_served():
    """Tables with room for 2^30 positions, of which few are used, and the most work that is counted in advance."""
    say("wide tables")
    for n, heads in ((64, 16), (1, 16), (1, 200)):
        b = Batch([(n, 200)], heads, heads, 16, 1024, "f16", "f16", seed=heads)
        table = torch.zeros((1, 2 ** 20), dtype=torch.int32, device="cuda")
        table[:, :b.table.shape[1]] = b.table
        b.check(b.run())
        b.table = table
        b.check(b.run())
    b = Batch([(1, 200)], 512, 512, 16, 1024, "f16", "f16")
    b.table = table
    with pytest.raises(L.LSCDError) as e:
        b.run()
    assert e.value.status == L.LSCD_ERROR_NOT_SUPPORTED


def test_starts_that_do_not_ascend():
    """Sequences that name the same tokens again and again, with more work than 31 bits count: the call ends, writes
    nothing outside its rows, and the next one is right."""
    say("starts that do not ascend")
    T, S, pages = 4096, 4096, 1024
    b = Batch([(T, 5000)], 16, 16, 16, 1024, "f16", "f16", seed=2)
    clean = b.run()
    start, length, table = b.start, b.length, b.table
    b.start = torch.tensor([0, T] * (S // 2) + [0], dtype=torch.int32, device="cuda")
    b.length = torch.full((S,), 2 ** 30, dtype=torch.int32, device="cuda")
    b.table = torch.zeros((S, pages), dtype=torch.int32, device="cuda")
    wide = torch.full((T + 2, 16, 16), 3.0, dtype=torch.float16, device="cuda")
    b.run(out=wide[1:-1])
    assert (wide[0] == 3).all() and (wide[-1] == 3).all()
    b.start, b.length, b.table = start, length, table
    assert torch.equal(b.run(), clean)


def test_strides_of_single_elements_do_not_count():
    """One sequence's length, one slot and a table of one column may have any stride there."""
    say("strides of single elements")
    b = Batch([(1, 10)], 4, 2, 64, 16, "f16", "f16", seed=4)
    want = b.run()
    b.length = torch.tensor([10, 99, 99], dtype=torch.int32, device="cuda")[::2][:1]
    b.table = torch.stack([b.table[:, 0], b.table[:, 0] + 1], 1)[:, ::2]
    assert torch.equal(b.run(), want)
    slot = torch.tensor([3, 99, 99], dtype=torch.int32, device="cuda")[::2][:1]
    k, v = (torch.randn((1, 2, 64), device="cuda").half() for _ in range(2))
    L.lscd_cache_write(b.cache(), k, v, slot)
    out = [torch.empty_like(k) for _ in range(2)]
    L.lscd_cache_read(b.cache(), slot, *out)
    assert torch.equal(out[0], k) and torch.equal(out[1], v)
    for t in (torch.arange(4, dtype=torch.int32, device="cuda")[::2], torch.zeros((1, 4), dtype=torch.int32, device="cuda")[:, ::2]):
        with pytest.raises(ValueError):
            L._ints(t, "t", t.device, t.dim())


def test_contents_out_of_range_are_those_of_the_nearest_range():
    """Lengths past the table, negative ones, pages outside the pool, starts outside the tokens: the result of the
    clamped arrays, and nothing written beside the output's rows."""
    say("clamped contents, compared")
    for n, dim in ((1, 64), (50, 64), (50, 256)):
        b = Batch([(n, 60), (n, 30), (n, 17)], 4, 2, dim, 16, "f16", "f16", seed=3)
        wide = torch.full((b.T + 2, 4, dim), 3.0, dtype=torch.float16, device="cuda")
        keep = b.start.clone(), b.length.clone(), b.table.clone()
        b.length[0], b.length[2] = 2 ** 31 - 1, -5
        b.table[0, -1], b.table[1, 0], b.table[1, 1] = -2 ** 31, 2 ** 31 - 1, b.pages
        b.start[0], b.start[3] = -7, 2 ** 31 - 1
        b.run(out=wide[1:-1])
        b.start, b.length, b.table = (x.clone() for x in keep)
        b.length[0], b.length[2] = b.table.shape[1] * 16, 0
        b.table[0, b.table[0] < 0] = 0
        b.table[1, 0], b.table[1, 1] = 0, 0
        assert torch.equal(wide[1:-1], b.run())
        assert (wide[0] == 3).all() and (wide[-1] == 3).all()


@pytest.mark.parametrize("kind,cache", [("f16", "e4m3"), ("bf16", "bf16")])
@pytest.mark.parametrize("heads,kv,dim", [(2, 2, 16), (6, 3, 32), (2, 1, 48), (4, 2, 96), (2, 2, 112), (2, 1, 144), (3, 1, 192),
                                          (2, 2, 240), (8, 1, 256)])
def test_head_sizes(heads, kv, dim, kind, cache):
    """Sizes between those of the other tests, decoding and in chunks."""
    say("head sizes", heads, kv, dim, kind, cache)
    for seqs in ([(1, 300), (2, 77), (1, 1)], [(70, 200), (0, 9), (33, 33), (1, 150)]):
        b = Batch(seqs, heads, kv, dim, 16, kind, cache, seed=dim)
        b.check(b.run())
        b.check(b.run(window=50), window=50)


@pytest.mark.parametrize("kind,cache", [("f16", "f16"), ("bf16", "e4m3")])
def test_many_sequences_of_both_kinds(kind, cache):
    """More than 64 sequences, those of few rows and of many among each other and in every block of 64."""
    say("many sequences", kind, cache)
    rng = np.random.default_rng(5)
    new = rng.choice([0, 1, 1, 3, 9, 20, 40, 70], 150)
    seqs = [(int(n), int(n + rng.integers(0, 90))) for n in new]
    seqs[10] = (1, 2500)
    seqs[140] = (40, 2000)
    b = Batch(seqs, 4, 2, 64, 16, kind, cache, seed=6)
    out = b.run()
    b.check(out)
    for _ in range(2):
        assert torch.equal(b.run(), out)
    only = Batch([(max(20, n), length + 20) for n, length in seqs], 4, 2, 64, 16, kind, cache, seed=7)
    only.check(only.run(window=33), window=33)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("heads,length", [(1, 33000), (1, 131072), (8, 70000)])
def test_an_item_of_many_parts(kind, heads, length):
    """One sequence whose positions go to more workgroups (74, 145 and 39) than are joined at a time, its scores
    climbing so that every batch of parts rescales those before it."""
    say("an item of many parts", kind, heads, length)
    b = Batch([(1, length)], heads, 1, 64, 1024, kind, kind, seed=heads)
    b.tensors[0].mul_(0.1)
    pages = b.table[0, :-(-length // 1024)].long()
    climb = (torch.arange(pages.numel() * 1024, device="cuda") * (30.0 / length)).view(-1, 1024)
    b.tensors[0][pages, 0, :, 0] = climb.to(b.q.dtype)
    b.q[:, :, 0] = 8.0
    out = b.run()
    q, k, v = b.q[0].double().cpu(), torch.from_numpy(b.values(0, 0))[:, 0], torch.from_numpy(b.values(1, 0))[:, 0]
    s = (q @ k.t()) * 64 ** -0.5
    w = torch.softmax(s, 1)
    o, a = w @ v, w @ v.abs()
    u, big = sv.ROUNDOFF[kind], ((q.abs() @ k.abs().t()) * 64 ** -0.5).amax(1, keepdim=True)
    e = 2 * (64 + 8) * 2.0 ** -24 * big + 2.0 ** -18
    small = 2.0 ** -32 * v.abs().sum(0) / torch.exp(s - s.amax(1, keepdim=True)).sum(1, keepdim=True) if kind == "f16" else 0.0
    assert ((out[0].double().cpu() - o).abs() <= u * o.abs() + (u + e) * a + small + sv.TINY[kind]).all()
    for _ in range(3):
        assert torch.equal(b.run(), out)
