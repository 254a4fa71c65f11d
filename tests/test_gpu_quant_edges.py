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
