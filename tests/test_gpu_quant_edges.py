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
