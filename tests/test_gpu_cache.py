"""The paged cache on the GPU, bit for bit against the plain definition.

* codes and scales of lscd_cache_write over types, head sizes, page sizes, strides, slot orders;
* what is not written stays; tokens without a slot are skipped, numbers past the cache too;
* lscd_cache_read gives code * scale rounded once, zeros without a slot;
* infinities, NaN, zeros, subnormals and vectors on both sides of a power-of-two step;
* streams, graphs, a pool whose element offsets pass 2^31, refusals.
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


def pool(pages, heads, page, dim, kind, seed):
    g = torch.Generator().manual_seed(seed)
    if kind == "e4m3":
        codes = [torch.randint(0, 127, (pages, heads, page, dim), generator=g, dtype=torch.uint8) for _ in range(2)]
        scales = [torch.exp2(torch.randint(-9, 9, (pages, heads, page), generator=g).float()) for _ in range(2)]
        return [x.cuda().view(torch.float8_e4m3fn) for x in codes] + [x.cuda() for x in scales]
    return [torch.randn((pages, heads, page, dim), generator=g).to(TYPES[kind]).cuda() for _ in range(2)] + [None, None]


def host(x):
    if x is None:
        return None
    return x.view(torch.uint8).cpu().numpy().copy() if x.dtype == torch.float8_e4m3fn else x.cpu().double().numpy()


def expect_write(new, slots, codes, scales, page):
    codes, scales = codes.copy(), scales.copy()
    for t, s in enumerate(slots):
        if 0 <= s < codes.shape[0] * page:
            for h in range(codes.shape[1]):
                x = new[t, h]
                scales[s // page, h, s % page] = sv.cache_scale(x)
                codes[s // page, h, s % page] = sv.e4m3_codes(x / sv.cache_scale(x))
    return codes, scales


@pytest.mark.parametrize("T,heads,dim,page,kind", [
    (1, 1, 16, 16, "f16"), (1, 96, 128, 16, "f16"), (17, 3, 64, 16, "bf16"), (40, 5, 80, 32, "f16"),
    (33, 2, 256, 64, "bf16"), (300, 4, 128, 128, "f16"), (19, 7, 112, 16, "bf16"), (20, 6, 48, 1024, "f16")])
def test_write_e4m3(T, heads, dim, page, kind):
    say(f"write T={T} heads={heads} dim={dim} page={page} {kind}")
    pages = (T + page - 1) // page + 2
    rng = np.random.default_rng(T * heads + dim)
    c = pool(pages, heads, page, dim, "e4m3", T)
    before = [host(x) for x in c]
    x = torch.from_numpy(rng.standard_normal((T, 3, heads, dim)) * np.exp(2 * rng.standard_normal((T, 3, heads, 1)))).to(TYPES[kind]).cuda()
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[rng.random(T) < 0.2] = -1
    if T > 2:
        slots[1], slots[2] = pages * page, 2 ** 31 - 1      # past the cache
    L.lscd_cache_write(L.Cache(*c), x[:, 1], x[:, 2], torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    for i in range(2):
        codes, scales = expect_write(x[:, 1 + i].cpu().double().numpy(), slots, before[i], before[2 + i], page)
        assert np.array_equal(host(c[i]), codes)
        assert np.array_equal(host(c[2 + i]), scales)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_write_special_values(kind):
    """Steps of the scale at 448 * 2^e, zeros, subnormals, infinities and NaN; ties of the rounding."""
    say("write special", kind)
    dim, page = 16, 16
    rows = [np.zeros(dim), np.full(dim, 448.0), np.full(dim, 449.0 if kind == "f16" else 450.0), np.full(dim, 1.75),
            np.full(dim, 1.7578125), np.linspace(-1, 1, dim), np.full(dim, 2.0 ** -24 if kind == "f16" else 2.0 ** -133),
            np.full(dim, 65504.0 if kind == "f16" else 3.0e38), np.full(dim, -0.0)]
    rows.append(np.where(np.arange(dim) == 3, np.inf, 2.0))
    rows.append(np.where(np.arange(dim) == 5, -np.inf, 300.0))
    rows.append(np.where(np.arange(dim) == 0, np.nan, np.arange(dim)))
    rows.append(np.full(dim, np.nan))
    rows.append(np.concatenate([[448.0], np.arange(1, dim) * 2.0 ** -10]))   # ties among the subnormal codes
    rows.append(np.concatenate([[256.0], 17 + 2 * np.arange(1, dim)]))       # ties among the normal ones
    x = torch.from_numpy(np.stack(rows))[:, None].to(TYPES[kind]).cuda()
    T = len(rows)
    c = pool(2, 1, page, dim, "e4m3", 5)
    before = [host(t) for t in c]
    slots = np.arange(T, dtype=np.int32) + 7
    L.lscd_cache_write(L.Cache(*c), x, x, torch.from_numpy(slots).cuda())
    codes, scales = expect_write(x.cpu().double().numpy(), slots, before[0], before[2], page)
    got = host(c[0])
    nan = (codes & 127) == 127
    assert np.array_equal((got & 127) == 127, nan)          # a NaN's sign says nothing
    assert np.array_equal(got[~nan], codes[~nan])
    assert np.array_equal(host(c[2]), scales)


@pytest.mark.parametrize("T,heads,dim,page,kind", [
    (1, 1, 16, 16, "f16"), (50, 3, 80, 16, "bf16"), (130, 56, 128, 64, "f16"), (9, 2, 256, 32, "bf16"), (21, 6, 64, 16, "f16")])
def test_read_e4m3(T, heads, dim, page, kind):
    say(f"read T={T} heads={heads} dim={dim} page={page} {kind}")
    rng = np.random.default_rng(T + dim)
    c = pool(4, heads, page, dim, "e4m3", T)
    slots = rng.integers(0, 4 * page, T).astype(np.int32)
    slots[T // 2] = -3
    if T > 3:
        slots[0] = 4 * page
    wide = torch.full((2, T, heads + 1, dim), 7.0, dtype=TYPES[kind], device="cuda")     # rows with a gap between
    L.lscd_cache_read(L.Cache(*c), torch.from_numpy(slots).cuda(), wide[0, :, :heads], wide[1, :, :heads])
    values = sv.e4m3_values()
    for i in range(2):
        codes, scales = host(c[i]), host(c[2 + i])
        want = np.zeros((T, heads, dim))
        for t, s in enumerate(slots):
            if 0 <= s < 4 * page:
                want[t] = values[codes[s // page, :, s % page]] * scales[s // page, :, s % page, None]
        assert torch.equal(wide[i, :, :heads].cpu(), torch.from_numpy(want).to(TYPES[kind]))
        assert (wide[i, :, heads] == 7.0).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_sixteen_bit_round_trip(kind):
    say("16-bit round trip", kind)
    T, heads, dim, page = 45, 3, 96, 16
    c = pool(5, heads, page, dim, kind, 3)
    before = [x.clone() for x in c[:2]]
    g = torch.Generator().manual_seed(1)
    k, v = (torch.randn((T, heads, dim), generator=g).to(TYPES[kind]).cuda() for _ in range(2))
    k[3, 1, 5], v[4, 0, 0] = float("inf"), float("nan")
    slots = torch.randperm(5 * page, generator=g)[:T].to(torch.int32).cuda()
    cache = L.Cache(c[0], c[1])
    L.lscd_cache_write(cache, k, v, slots)
    ko, vo = torch.empty_like(k), torch.empty_like(v)
    L.lscd_cache_read(cache, slots, ko, vo)
    assert torch.equal(ko.view(torch.int16), k.view(torch.int16)) and torch.equal(vo.view(torch.int16), v.view(torch.int16))
    rest = torch.ones(5 * page, dtype=torch.bool)
    rest[slots.cpu().long()] = False
    for a, b in zip(c[:2], before):
        flat = lambda x: x.permute(0, 2, 1, 3).reshape(5 * page, heads, dim)[rest.to(x.device)]  # noqa: E731
        assert torch.equal(flat(a), flat(b))


def test_offsets_past_32_bits():
    """A pool of 2.2e9 values: the last page's elements lie past 2^31."""
    say("large pool")
    heads, page, dim = 8, 16, 128
    pages = (2 ** 31 + 2 ** 27) // (heads * page * dim)
    k = torch.zeros((pages, heads, page, dim), dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    ks, vs = (torch.ones((pages, heads, page), device="cuda") for _ in range(2))
    x = torch.randn((3, heads, dim), device="cuda").half()
    slots = torch.tensor([pages * page - 1, 0, (pages - 1) * page], dtype=torch.int32, device="cuda")
    cache = L.Cache(k, v, ks, vs)
    L.lscd_cache_write(cache, x, -x, slots)
    a, b = torch.empty_like(x), torch.empty_like(x)
    L.lscd_cache_read(cache, slots, a, b)
    want = x.cpu().double().numpy()
    scale = np.array([[sv.cache_scale(want[t, h]) for h in range(heads)] for t in range(3)])[..., None]
    want = sv.e4m3_values()[sv.e4m3_codes(want / scale)] * scale
    assert np.array_equal(a.cpu().double().numpy(), want) and np.array_equal(b.cpu().double().numpy(), -want)
    assert int((k[1:pages - 1].view(torch.uint8) != 0).any()) == 0


def test_stream_graph_and_nothing_to_do():
    say("cache on a stream, in a graph")
    c = pool(4, 2, 16, 64, "e4m3", 9)
    cache = L.Cache(*c)
    x = torch.randn((10, 2, 64), device="cuda").half()
    slots = torch.arange(10, dtype=torch.int32, device="cuda")
    out = [torch.empty_like(x) for _ in range(2)]
    L.lscd_cache_write(cache, x[:0], x[:0], slots[:0])
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.lscd_cache_write(cache, x, x, slots)
        L.lscd_cache_read(cache, slots, *out)
    s.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lscd_cache_write(cache, x, x, slots)
        L.lscd_cache_read(cache, slots, *out)
    for seed in range(3):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)).half())
        graph.replay()
        torch.cuda.synchronize()
        got = [t.clone() for t in out]
        L.lscd_cache_write(cache, x, x, slots)
        L.lscd_cache_read(cache, slots, *out)
        torch.cuda.synchronize()
        assert torch.equal(got[0], out[0]) and torch.equal(got[1], out[1]) and torch.equal(out[0], out[1])


def test_refusals():
    say("cache refusals")
    k = torch.zeros((3, 2, 16, 64), dtype=torch.float8_e4m3fn, device="cuda")
    sc = torch.ones((3, 2, 16), device="cuda")
    x = torch.zeros((4, 2, 64), device="cuda", dtype=torch.float16)
    slots = torch.zeros(4, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        L.Cache(k, k)                                       # no scales
    with pytest.raises(ValueError):
        L.Cache(x[None], x[None], sc, sc)                   # scales of a 16-bit cache
    with pytest.raises(ValueError):
        L.Cache(k, k[:, :, :, :32], sc, sc)
    good = L.Cache(k, k.clone(), sc, sc.clone())
    with pytest.raises(ValueError):
        L.lscd_cache_write(good, x, x, slots[:3])
    with pytest.raises(ValueError):
        L.lscd_cache_write(good, x, x, slots.long())
    with pytest.raises(ValueError):
        L.lscd_cache_write(good, x, x.bfloat16(), slots)
    with pytest.raises(ValueError):
        L.lscd_cache_write(good, x[:, :, ::2], x, slots)

    def status(fn, *args):
        with pytest.raises(L.LSCDError) as e:
            fn(*args)
        return e.value.status

    odd = torch.zeros((3, 2, 24, 64), dtype=torch.float16, device="cuda")
    assert status(L.lscd_cache_write, L.Cache(odd, odd), x, x, slots) == L.LSCD_ERROR_NOT_SUPPORTED   # page of 24
    odd = torch.zeros((3, 2, 16, 40), dtype=torch.float16, device="cuda")
    assert status(L.lscd_cache_write, L.Cache(odd, odd), x[:, :, :40].contiguous(), x[:, :, :40].contiguous(), slots) == \
        L.LSCD_ERROR_NOT_SUPPORTED                                                                     # heads of 40
    b = torch.zeros((3, 2, 16, 64), dtype=torch.bfloat16, device="cuda")
    assert status(L.lscd_cache_write, L.Cache(b, b), x, x, slots) == L.LSCD_ERROR_NOT_SUPPORTED        # types
    shifted = torch.zeros(4 * 128 + 1, dtype=torch.float16, device="cuda")[1:].view(4, 2, 64)
    assert status(L.lscd_cache_write, good, shifted, x, slots) == L.LSCD_ERROR_INVALID_VALUE           # alignment
    strided = torch.zeros((4, 132), dtype=torch.float16, device="cuda")[:, :128].view(4, 2, 64)
    assert status(L.lscd_cache_read, good, slots, strided, x) == L.LSCD_ERROR_INVALID_VALUE            # stride
