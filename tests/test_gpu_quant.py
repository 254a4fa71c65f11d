"""The product with 4-bit codes on the GPU against the plain 64-bit definition.

Tolerance, per value, from the arithmetic: u |y| for the output's rounding, and for fp32 sums of K
exact terms in any order and G scaled group sums (K + 2 G + 8) 2^-24 of the sum of the terms'
magnitudes: |(c - z) x s| in float16, and in bfloat16 ((16 + c) + (16 + z)) |x s|, whose difference is
taken after summing.  Whole-number cases whose sums are exact have to be equal.
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


def matrix(M, K, group, zeros, kind, seed, whole=False):
    rng = np.random.default_rng(seed)
    G = -(-K // group)
    codes = rng.integers(0, 256, (M, (K + 1) // 2)).astype(np.uint8)
    s = 2.0 ** rng.integers(-2, 2, (M, G)) if whole else np.exp(rng.standard_normal((M, G)) - 4)
    scales = torch.from_numpy(s).to(TYPES[kind]).cuda()
    z = rng.integers(0, 16, (M, G)).astype(np.uint8) if zeros else None
    h = L.lscd_quant_encode(torch.from_numpy(codes).cuda(), scales, K, None if z is None else torch.from_numpy(z).cuda(), group)
    return h, *sv.quant_weights(codes, scales.cpu().double().numpy(), z, K, group), z


def check(y, x, c, s, z, kind, group):
    x = x.cpu().double().numpy()
    w, K = c * s, c.shape[1]
    want = x @ w.T
    off = 0 if kind == "f16" else 47 + np.abs(c)            # (16 + c) + (16 + z) <= 47 + |c - z|
    terms = np.abs(x) @ ((np.abs(c) + off) * s).T
    tol = sv.ROUNDOFF[kind] * np.abs(want) + (K + 2 * -(-K // group) + 8) * 2.0 ** -24 * terms + sv.TINY[kind]
    d = np.abs(y.cpu().double().numpy() - want)
    assert (d <= tol).all(), float((d / tol).max())


SHAPES = [(1, 1, 1), (16, 128, 16), (17, 129, 3), (64, 1024, 1), (100, 640, 7), (333, 1000, 16), (48, 4099, 5), (1000, 555, 33),
          (130, 2048, 64), (70, 900, 48), (2100, 384, 17), (40, 8192, 2)]


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True), (256, False)])
@pytest.mark.parametrize("M,K,N", SHAPES)
def test_product(M, K, N, group, zeros, kind):
    say(f"quant {M}x{K} N={N} group={group} zeros={zeros} {kind}")
    h, c, s, z = matrix(M, K, group, zeros, kind, M + K + N)
    x = torch.from_numpy(np.random.default_rng(N).standard_normal((N, K))).to(TYPES[kind]).cuda()
    y = torch.full((N, M), float("nan"), dtype=TYPES[kind], device="cuda")
    L.lscd_quant_linear(h, x, y)
    check(y, x, c, s, z, kind, group)
    again = torch.empty_like(y)
    for _ in range(2):
        L.lscd_quant_linear(h, x, again)
        assert torch.equal(again, y)


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(12288, 2048, 1), (3000, 12288, 16), (512, 16384, 64), (4100, 4096, 20), (8200, 1024, 4)])
def test_larger(M, K, N, kind):
    """Sizes that fill the GPU in each direction, against a product in 64 bits on the GPU."""
    say(f"quant {M}x{K} N={N} {kind}")
    g = torch.Generator(device="cuda").manual_seed(M)
    G = K // 128
    codes = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.exp(torch.randn((M, G), generator=g, device="cuda") - 4).to(TYPES[kind])
    zeros = torch.randint(0, 16, (M, G), generator=g, device="cuda", dtype=torch.uint8)
    x = torch.randn((N, K), generator=g, device="cuda").to(TYPES[kind])
    h = L.lscd_quant_encode(codes, scales, K, zeros, 128)
    y = torch.full((N, M), float("nan"), dtype=TYPES[kind], device="cuda")
    L.lscd_quant_linear(h, x, y)
    c = torch.stack([codes & 15, codes >> 4], 2).flatten(1).double() - zeros.double().repeat_interleave(128, 1)
    s = scales.double().repeat_interleave(128, 1)
    want = x.double() @ (c * s).t()
    terms = x.double().abs() @ ((c.abs() + (0 if kind == "f16" else 47 + c.abs())) * s).t()
    tol = sv.ROUNDOFF[kind] * want.abs() + (K + 2 * G + 8) * 2.0 ** -24 * terms + sv.TINY[kind]
    assert ((y.double() - want).abs() <= tol).all()


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("N", [1, 16, 33, 65, 150])
def test_whole_numbers_are_exact(kind, N):
    """Small whole x, scales powers of two: every sum is exact in fp32, so y is the rounded result."""
    say("quant whole numbers", kind, N)
    h, c, s, z = matrix(200, 1100, 64, True, kind, N, whole=True)
    x = torch.from_numpy(np.random.default_rng(N).integers(-2, 3, (N, 1100)).astype(np.float64)).to(TYPES[kind]).cuda()
    y = torch.empty((N, 200), dtype=TYPES[kind], device="cuda")
    L.lscd_quant_linear(h, x, y)
    want = torch.from_numpy(x.cpu().double().numpy() @ (c * s).T).to(TYPES[kind])
    assert torch.equal(y.cpu(), want)


@pytest.mark.parametrize("M,K", [(1689, 1645), (3974, 8557)])
def test_every_number_of_tokens(M, K):
    """Each number of tokens has its own plan, and fewer tokens may split K into more ranges: the partial
    sums' room has to hold every plan's (whole numbers: the results are exact, as above)."""
    say("quant every number of tokens", M, K)
    h, c, s, z = matrix(M, K, 128, True, "f16", M, whole=True)
    x = torch.from_numpy(np.random.default_rng(K).integers(-2, 3, (64, K)).astype(np.float64)).half().cuda()
    want = torch.from_numpy(x.cpu().double().numpy() @ (c * s).T).half()
    for N in range(1, 65):
        y = torch.full((N, M), float("nan"), dtype=torch.float16, device="cuda")
        L.lscd_quant_linear(h, x[:N], y)
        assert torch.equal(y.cpu(), want[:N]), N


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("group", [32, 64, 128, 384])
def test_decode(kind, group):
    say("quant decode", kind, group)
    h, c, s, z = matrix(37, 1003, group, True, kind, 5)
    w = torch.empty((37, 1003), dtype=TYPES[kind], device="cuda")
    L.lscd_quant_decode(h, w)
    want = torch.from_numpy(c * s).float()                   # code x scale is exact in fp32
    assert torch.equal(w.cpu(), want.to(TYPES[kind]))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
def test_strides_and_alignment(kind):
    """Rows of x and y inside wider tensors, at odd offsets; what lies between is neither read into y nor written."""
    say("quant strides", kind)
    M, K, N = 75, 515, 9
    h, c, s, z = matrix(M, K, 32, True, kind, 6)
    xw = torch.full((N, K + 7), float("nan"), dtype=TYPES[kind], device="cuda")
    x = xw[:, 3:3 + K]
    x.copy_(torch.randn((N, K)))
    yw = torch.full((N, M + 5), 3.0, dtype=TYPES[kind], device="cuda")
    L.lscd_quant_linear(h, x, yw[:, 1:1 + M])
    check(yw[:, 1:1 + M], x, c, s, z, kind, 32)
    assert (yw[:, 0] == 3).all() and (yw[:, 1 + M:] == 3).all()


def test_strides_of_single_rows_and_columns_do_not_count():
    """A matrix of one row, or of one byte a row, may have any stride in that direction."""
    say("quant single rows and columns")
    for M, K in ((1, 64), (40, 2)):
        rng = np.random.default_rng(M)
        codes = torch.from_numpy(rng.integers(0, 256, (M, K // 2)).astype(np.uint8)).cuda()
        scales = torch.ones((M, 1), dtype=torch.float16, device="cuda")
        x = torch.from_numpy(rng.integers(-2, 3, (3, K)).astype(np.float64)).half().cuda()
        odd = codes.as_strided(codes.shape, (1, 1) if M == 1 else (1, 7))
        y = [torch.empty((3, M), dtype=torch.float16, device="cuda") for _ in range(2)]
        for c, out in zip((codes, odd), y):
            L.lscd_quant_linear(L.lscd_quant_encode(c, scales, K, group=64), x, out)
        assert torch.equal(y[0], y[1])


def test_what_is_not_finite_stays_in_its_row():
    say("quant nan rows")
    h, c, s, z = matrix(90, 700, 128, True, "f16", 7)
    x = torch.randn((20, 700), device="cuda").half()
    y, clean = (torch.empty((20, 90), dtype=torch.float16, device="cuda") for _ in range(2))
    L.lscd_quant_linear(h, x, clean)
    x[3, 5], x[17, 699] = float("inf"), float("nan")
    L.lscd_quant_linear(h, x, y)
    keep = torch.tensor([i for i in range(20) if i not in (3, 17)], device="cuda")
    assert torch.equal(y[keep], clean[keep]) and not torch.isfinite(y[3]).any() and torch.isnan(y[17]).all()
    want = c[:, 5] * np.inf                                  # inf times code - zero: a sign, or NaN where they are equal
    got = y[3].cpu().double().numpy()
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(got[~np.isnan(got)], want[~np.isnan(want)])


def test_stream_and_graph():
    say("quant graph")
    for M, K, N in ((100, 4096, 3), (300, 8192, 40)):
        h, *_ = matrix(M, K, 128, False, "f16", 8)
        x = torch.randn((N, K), device="cuda").half()
        y, want = (torch.empty((N, M), dtype=torch.float16, device="cuda") for _ in range(2))
        L.lscd_quant_linear(h, x, want)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        L.lscd_quant_linear(h, x, y, stream=s)
        s.synchronize()
        assert torch.equal(y, want)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            L.lscd_quant_linear(h, x, y)
        for _ in range(4):
            x.normal_()
            graph.replay()
            L.lscd_quant_linear(h, x, want)
            torch.cuda.synchronize()
            assert torch.equal(y, want)


def test_nothing_to_do_and_refusals():
    say("quant refusals")
    codes = torch.zeros((32, 64), dtype=torch.uint8, device="cuda")
    scales = torch.ones((32, 1), dtype=torch.float16, device="cuda")
    h = L.lscd_quant_encode(codes, scales, 128)
    x, y = torch.zeros((2, 128), dtype=torch.float16, device="cuda"), torch.zeros((2, 32), dtype=torch.float16, device="cuda")
    L.lscd_quant_linear(h, x[:0], y[:0])
    for bad in (lambda: L.lscd_quant_linear(h, x[:, :64], y), lambda: L.lscd_quant_linear(h, x, y[:1]),
                lambda: L.lscd_quant_linear(h, x.bfloat16(), y), lambda: L.lscd_quant_linear(h, x, y.t().contiguous().t()),
                lambda: L.lscd_quant_encode(codes, scales, 130), lambda: L.lscd_quant_encode(codes, scales.float(), 128),
                lambda: L.lscd_quant_encode(codes, scales, 128, codes), lambda: L.lscd_quant_encode(codes, scales[:31], 128)):
        with pytest.raises(ValueError):
            bad()
    for group in (0, 16, 96, 200):
        G = -(-128 // group) if group else 0
        with pytest.raises(L.LSCDError) as e:
            L.lscd_quant_encode(codes, torch.ones((32, G), dtype=torch.float16, device="cuda"), 128, None, group)
        assert e.value.status == (L.LSCD_ERROR_NOT_SUPPORTED if group else L.LSCD_ERROR_INVALID_VALUE)
