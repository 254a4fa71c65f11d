"""The product with 4-bit codes at the ends of its types' ranges and sizes, and at long K.

Whole-number cases whose sums are exact in fp32 have to come out as the rounded result.
"""
import numpy as np
import pytest

from oracle import serving as sv
from tests._util import say
from tests.test_gpu_quant import TYPES, matrix

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

if torch.cuda.is_available():
    import unstructured_sparse_skinny_amd as L


@pytest.mark.parametrize("N", [1, 5, 20, 64])
@pytest.mark.parametrize("group,zeros", [(32, True), (128, False)])
@pytest.mark.parametrize("power", [126, 123, 119, 60, -100, -120, -126, -132])
def test_bfloat16_range(N, group, zeros, power):
    """x from the largest powers of two to subnormal ones; scales that bring y back to where it is finite."""
    say("quant bfloat16 range", N, group, zeros, power)
    rng = np.random.default_rng(N + group)
    M, K = 70, 640
    codes = rng.integers(0, 256, (M, K // 2)).astype(np.uint8)
    z = rng.integers(0, 16, (M, K // group)).astype(np.uint8) if zeros else None
    scales = torch.from_numpy(2.0 ** rng.integers(-17, -14, (M, K // group)) * (1.0 if power > 0 else 2.0 ** 16)).bfloat16().cuda()
    h = L.lscd_quant_encode(torch.from_numpy(codes).cuda(), scales, K, None if z is None else torch.from_numpy(z).cuda(), group)
    c, s = sv.quant_weights(codes, scales.cpu().double().numpy(), z, K, group)
    x = torch.from_numpy(rng.integers(-2, 3, (N, K)) * 2.0 ** (power - (1 if power > 0 else 0))).bfloat16().cuda()
    y = torch.full((N, M), float("nan"), dtype=torch.bfloat16, device="cuda")
    L.lscd_quant_linear(h, x, y)
    want = torch.from_numpy(x.cpu().double().numpy() @ (c * s).T).bfloat16()
    assert torch.isfinite(want).all() and torch.equal(y.cpu(), want)


def test_most_rows():
    """As many rows as are supported, every one of them right; one more is refused."""
    say("quant most rows")
    M, K = 2 ** 25, 3
    g = torch.Generator(device="cuda").manual_seed(1)
    codes = torch.randint(0, 256, (M + 1, 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.ones((M + 1, 1), dtype=torch.float16, device="cuda")
    with pytest.raises(L.LSCDError) as e:
        L.lscd_quant_encode(codes, scales, K)
    assert e.value.status == L.LSCD_ERROR_NOT_SUPPORTED
    h = L.lscd_quant_encode(codes[:M], scales[:M], K)
    w = (torch.stack([codes[:M] & 15, codes[:M] >> 4], 2).flatten(1)[:, :K].half() - 8)
    got = torch.full((M, K), 99.0, dtype=torch.float16, device="cuda")
    assert torch.equal(L.lscd_quant_decode(h, got), w)
    x = torch.tensor([[1.0, 2.0, -3.0], [5.0, 0.0, 1.0]], dtype=torch.float16, device="cuda")
    y = torch.full((2, M), 99.0, dtype=torch.float16, device="cuda")
    L.lscd_quant_linear(h, x, y)
    for n in range(2):
        assert torch.equal(y[n], sum(w[:, k] * x[n, k] for k in range(K)))


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("group,zeros", [(32, True), (64, False), (128, True)])
@pytest.mark.parametrize("M,K", [(300, 8192), (130, 16384), (77, 9001)])
def test_long_sums_are_exact(M, K, group, zeros, kind):
    """Whole x and power-of-two scales, sums of thousands of columns below 2^24 of their unit: every output is the
    rounded result, over splits of K, pipelines of many units, every form by tokens and several launches."""
    say("quant long sums", M, K, group, zeros, kind)
    h, c, s, z = matrix(M, K, group, zeros, kind, M, whole=True)
    x = torch.from_numpy(np.random.default_rng(K).integers(-2, 3, (200, K)).astype(np.float64)).to(TYPES[kind]).cuda()
    want = torch.from_numpy(x.cpu().double().numpy() @ (c * s).T).to(TYPES[kind])
    for N in (1, 2, 7, 16, 17, 32, 33, 64, 65, 130, 200):
        y = torch.full((N, M), float("nan"), dtype=TYPES[kind], device="cuda")
        L.lscd_quant_linear(h, x[:N], y)
        assert torch.equal(y.cpu(), want[:N]), N


@pytest.mark.parametrize("kind", ["f16", "bf16"])
@pytest.mark.parametrize("M,K,N", [(5003, 12288, 16), (2000, 16384, 64), (3000, 7168, 150)])
def test_error_of_random_sums(M, K, N, kind):
    """Random x and scales: the error's norm is that of y's rounding (steps of 2 u at fractions of 1 to 2: u / sqrt(3) =
    0.58 u of a value in the mean square at most) and of fp32 sums, whose rounding errors add up like a random walk:
    2^-24 sqrt(K + 2 G) of a typical partial sum, which is at most sqrt(2 x 47^2 / 21) of y's in bfloat16 (two sums of
    terms of up to 47 in place of one of terms of 21 in the mean square)."""
    say("quant error norm", M, K, N, kind)
    g = torch.Generator(device="cuda").manual_seed(K)
    G = K // 128
    codes = torch.randint(0, 256, (M, K // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = torch.exp(0.3 * torch.randn((M, G), generator=g, device="cuda") - 4).to(TYPES[kind])
    x = torch.randn((N, K), generator=g, device="cuda").to(TYPES[kind])
    y = torch.empty((N, M), dtype=TYPES[kind], device="cuda")
    L.lscd_quant_linear(L.lscd_quant_encode(codes, scales, K), x, y)
    w = (torch.stack([codes & 15, codes >> 4], 2).flatten(1).double() - 8) * scales.double().repeat_interleave(128, 1)
    want = x.double() @ w.t()
    error = float((y.double() - want).norm() / want.norm())
    assert error < 0.58 * sv.ROUNDOFF[kind] + 2.0 ** -24 * (K + 2 * G) ** 0.5 * (2 * 47 ** 2 / 21) ** 0.5
