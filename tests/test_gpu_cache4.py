"""The paged cache of 4-bit codes on the GPU, bit for bit against the plain definition.

* codes and scale bytes of lscd_cache_write over types, head sizes (whole groups of 32 channels and a half one),
  page sizes, slices of a wider tensor, slot orders; bytes that nobody owns stay;
* lscd_cache_read: code * scale rounded once, zeros without a slot, NaN under a scale byte of 255, any bytes;
* steps of the scale, ties, zeros of both signs, subnormals, the largest values, infinities and NaN;
* a stream, a replayed graph, a pool whose byte offsets pass 2^31, refusals.
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


def pool4(pages, heads, page, dim, seed, low=110, high=140):
    """k, v, k_scale, v_scale with random codes and scales 2^(low - 127) and up."""
    g = torch.Generator().manual_seed(seed)
    codes = [torch.randint(0, 256, (pages, heads, page, dim // 2), generator=g, dtype=torch.uint8) for _ in range(2)]
    row = 2 if dim <= 64 else 4 if dim <= 128 else 8
    scales = [torch.randint(low, high, (pages, heads, page, row), generator=g, dtype=torch.uint8) for _ in range(2)]
    return [x.cuda() for x in codes + scales]


def expect(new, slots, codes, scales, page):
    """The pool after a write; codes of groups that are not finite as they were (they say nothing)."""
    codes, scales = codes.copy(), scales.copy()
    for t, s in enumerate(slots):
        if not 0 <= s < codes.shape[0] * page:
            continue
        for h in range(codes.shape[1]):
            for a in range(0, new.shape[2], 32):
                c, byte = sv.e2m1_group(new[t, h, a:a + 32])
                scales[s // page, h, s % page, a // 32] = byte
                if c is not None:
                    codes[s // page, h, s % page, a // 2:a // 2 + len(c) // 2] = c[0::2] | c[1::2] << 4
    return codes, scales


@pytest.mark.parametrize("T,heads,dim,page,kind", [
    (1, 1, 16, 16, "f16"), (1, 96, 128, 16, "f16"), (17, 3, 64, 16, "bf16"), (40, 5, 80, 32, "f16"), (5, 2, 32, 16, "bf16"),
    (33, 2, 256, 64, "bf16"), (150, 4, 128, 128, "f16"), (19, 7, 112, 16, "bf16"), (20, 6, 48, 1024, "f16"), (9, 2, 144, 16, "f16")])
def test_write(T, heads, dim, page, kind):
    say(f"write T={T} heads={heads} dim={dim} page={page} {kind}")
    pages = (T + page - 1) // page + 2
    rng = np.random.default_rng(T * heads + dim)
    c = pool4(pages, heads, page, dim, T)
    before = [x.cpu().numpy().copy() for x in c]
    x = rng.standard_normal((T, 3, heads, dim)) * np.exp(2 * rng.standard_normal((T, 3, heads, dim // 16, 1))).repeat(16, 4).reshape(T, 3, heads, dim)
    x = torch.from_numpy(x).to(TYPES[kind]).cuda()
    slots = rng.permutation(pages * page)[:T].astype(np.int32)
    slots[rng.random(T) < 0.2] = -1
    if T > 2:
        slots[1], slots[2] = pages * page, 2 ** 31 - 1      # past the cache
    L.lscd_cache_write(L.Cache(*c), x[:, 1], x[:, 2], torch.from_numpy(slots).cuda())
    torch.cuda.synchronize()
    for i in range(2):
        codes, scales = expect(x[:, 1 + i].cpu().double().numpy(), slots, before[i], before[2 + i], page)
        assert np.array_equal(c[2 + i].cpu().numpy(), scales)
        assert np.array_equal(c[i].cpu().numpy(), codes)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_write_special_values(kind):
    say("write special", kind)
    dim, page = 32, 16
    tiny = 2.0 ** -24 if kind == "f16" else 2.0 ** -133
    rows = [np.zeros(dim), np.full(dim, -0.0), np.full(dim, 6.0), np.full(dim, 6.03125), np.full(dim, -3.0), np.full(dim, 3.015625),
            np.linspace(-1, 1, dim), np.full(dim, tiny), np.full(dim, 65504.0 if kind == "f16" else 3.38e38),
            np.concatenate([[6.0], np.arange(1, dim) * 0.25]),                                # every tie between two codes
            np.concatenate([[-6.0], np.arange(1, dim) * -0.125]), np.concatenate([[6 * 2.0 ** -10], np.arange(1, dim) * tiny]),
            np.where(np.arange(dim) == 31, 1e-3, 0.0)]
    rows += [np.where(np.arange(dim) == 3, np.inf, 2.0), np.where(np.arange(dim) == 30, -np.inf, 300.0),
             np.where(np.arange(dim) == 0, np.nan, np.arange(dim)), np.full(dim, np.nan)]
    x = torch.from_numpy(np.stack(rows))[:, None].to(TYPES[kind])
    x = torch.cat([x, x.flip(0)], dim=2).cuda()               # two groups: what is not finite in one leaves the other
    T, c = len(rows), pool4(3, 1, page, 2 * dim, 5)
    before = [t.cpu().numpy().copy() for t in c]
    slots = np.arange(T, dtype=np.int32) + 7
    L.lscd_cache_write(L.Cache(*c), x, x, torch.from_numpy(slots).cuda())
    codes, scales = expect(x.cpu().double().numpy(), slots, before[0], before[2], page)
    finite = np.repeat(scales != 255, 16, axis=-1)
    assert np.array_equal(c[2].cpu().numpy(), scales)
    assert np.array_equal(c[0].cpu().numpy()[finite], codes[finite])
    got = [torch.empty_like(x) for _ in range(2)]
    L.lscd_cache_read(L.Cache(*c), torch.from_numpy(slots).cuda(), *got)
    want = torch.from_numpy(sv.e2m1_values(codes, scales, 2 * dim)).permute(0, 2, 1, 3).reshape(-1, 1, 2 * dim)[7:7 + T].to(TYPES[kind])
    assert torch.equal(torch.isnan(got[1].cpu()), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(got[0].cpu(), 7.0), torch.nan_to_num(want, 7.0))


@pytest.mark.parametrize("T,heads,dim,page,kind", [
    (1, 1, 16, 16, "f16"), (50, 3, 80, 16, "bf16"), (130, 56, 128, 64, "f16"), (9, 2, 256, 32, "bf16"), (21, 6, 64, 16, "f16"),
    (7, 2, 240, 16, "f16")])
def test_read(T, heads, dim, page, kind):
    """Every scale byte, subnormal results and those past the type's largest among them."""
    say(f"read T={T} heads={heads} dim={dim} page={page} {kind}")
    rng = np.random.default_rng(T + dim)
    c = pool4(4, heads, page, dim, T, 0, 256)
    slots = rng.integers(0, 4 * page, T).astype(np.int32)
    slots[T // 2] = -3
    if T > 3:
        slots[0] = 4 * page
    wide = torch.full((2, T, heads + 1, dim), 7.0, dtype=TYPES[kind], device="cuda")     # rows with a gap between
    L.lscd_cache_read(L.Cache(*c), torch.from_numpy(slots).cuda(), wide[0, :, :heads], wide[1, :, :heads])
    for i in range(2):
        values = sv.e2m1_values(c[i].cpu().numpy(), c[2 + i].cpu().numpy(), dim)
        want = np.zeros((T, heads, dim))
        for t, s in enumerate(slots):
            if 0 <= s < 4 * page:
                want[t] = values[s // page, :, s % page]
        want = torch.from_numpy(want).to(TYPES[kind])
        got = wide[i, :, :heads].cpu()
        assert torch.equal(torch.isnan(got), torch.isnan(want))
        assert torch.equal(torch.nan_to_num(got, 7.0, 9.0, -9.0), torch.nan_to_num(want, 7.0, 9.0, -9.0))
        assert (wide[i, :, heads] == 7.0).all()


def test_offsets_past_32_bits():
    """Pages at the end of a pool of more than 2^31 bytes of codes."""
    say("large pool")
    heads, page, dim = 8, 16, 128
    pages = (2 ** 31 + 2 ** 27) // (heads * page * dim // 2)
    c = [torch.zeros((pages, heads, page, dim // 2), dtype=torch.uint8, device="cuda") for _ in range(2)]
    c += [torch.full((pages, heads, page, 4), 127, dtype=torch.uint8, device="cuda") for _ in range(2)]
    x = torch.randn((4, heads, dim), device="cuda").half()
    slots = torch.tensor([pages * page - 1, 3, pages * page - 17, pages * page // 2], dtype=torch.int32, device="cuda")
    L.lscd_cache_write(L.Cache(*c), x, -x, slots)
    got = [torch.empty_like(x) for _ in range(2)]
    L.lscd_cache_read(L.Cache(*c), slots, *got)
    want = torch.zeros((4, heads, dim))
    for t in range(4):
        for h in range(heads):
            for a in range(0, dim, 32):
                code, byte = sv.e2m1_group(x[t, h, a:a + 32].cpu().double().numpy())
                want[t, h, a:a + 32] = torch.from_numpy(np.where(code > 7, -1, 1) * sv.E2M1[code & 7] * 2.0 ** (byte - 127))
    assert torch.equal(got[0].cpu().float(), want) and torch.equal(got[1].cpu().float(), -want)
    assert int((c[0].flatten(1) != 0).any(1).sum()) == 4          # nothing else was written


def test_stream_and_graph():
    say("stream, graph")
    c = pool4(6, 3, 16, 64, 1)
    cache = L.Cache(*c)
    k, v = (torch.randn((20, 3, 64), device="cuda").half() for _ in range(2))
    slots = torch.randperm(96, device="cuda")[:20].to(torch.int32)
    out = [torch.empty_like(k) for _ in range(2)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        L.lscd_cache_write(cache, k, v, slots)
        L.lscd_cache_read(cache, slots, *out)
    s.synchronize()
    want = [x.clone() for x in out]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        L.lscd_cache_write(cache, k, v, slots)
        L.lscd_cache_read(cache, slots, *out)
    for _ in range(3):
        for x in c:
            x.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    k.normal_()
    graph.replay()
    torch.cuda.synchronize()
    assert not torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_refusals():
    say("refusals")
    k, v, ks, vs = pool4(2, 2, 16, 80, 0)
    assert L.Cache(k, v, ks, vs).head_dim == 80
    for bad in ((k, v), (k, v, ks), (k, v, ks[..., :2], vs[..., :2]), (k, v, ks.to(torch.int8), vs.to(torch.int8)),
                (k, v, ks[..., 0].float(), vs[..., 0].float()), (k.view(torch.int8), v.view(torch.int8), ks, vs)):
        with pytest.raises(ValueError):
            L.Cache(*bad)
    x = torch.zeros((1, 2, 80), device="cuda").half()
    slot = torch.zeros(1, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        L.lscd_cache_write(L.Cache(k, v, ks, vs), x[..., :40], x[..., :40], slot)
    odd = pool4(2, 2, 16, 40, 0)                                  # 40 channels: not a multiple of 16
    with pytest.raises(L.LSCDError) as e:
        L.lscd_cache_write(L.Cache(*odd), x[..., :40].contiguous(), x[..., :40].contiguous(), slot)
    assert e.value.status == L.LSCD_ERROR_NOT_SUPPORTED
