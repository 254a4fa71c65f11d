"""What the serving operators refuse before they look at a device, and what their Python layer checks (CPU)."""
import ctypes

import pytest

import unstructured_sparse_skinny_amd as L


def encode(M, K, group=128, row_bytes=None):
    """Status of lscd_quant_encode for arrays that are not there: arguments that pass end at the missing device."""
    h = ctypes.c_void_p()
    rb = (K + 1) // 2 if row_bytes is None else row_bytes
    st = L._lib.lscd_quant_encode(0x1000, rb, 0x1000, None, M, K, group, L.LSCD_F16, None, ctypes.byref(h))
    assert not h.value
    return st


@pytest.mark.skipif(L.torch.cuda.is_available(), reason="sizes that pass would be read")
@pytest.mark.parametrize("M,K,ok", [
    (2 ** 25, 3, True), (2 ** 25 + 1, 3, False), (1, 2 ** 24, True), (1, 2 ** 24 + 1, False),
    (2 ** 15, 2 ** 22, False), (2 ** 15 - 16, 2 ** 22, True), (2 ** 25, 2 ** 12, False), (2 ** 14, 2 ** 23, False)])
def test_largest_matrices(M, K, ok):
    """A grid has fewer than 2^32 threads in a dimension: sizes whose launches would pass that are refused."""
    assert encode(M, K) == (L.LSCD_ERROR_HIP if ok else L.LSCD_ERROR_NOT_SUPPORTED)


def test_tensors_of_another_device_are_refused(monkeypatch):
    """Every call of the Python layer asks for its stream with its tensors' device."""
    monkeypatch.setattr(L, "_current_device", lambda: 0)
    monkeypatch.setattr(L, "_current_raw_stream", lambda index: 70 + index)
    here, other = L.torch.device("cuda", 0), L.torch.device("cuda", 1)
    assert L._stream_on(None, here) == 70 and L._stream_on(5, here) == 5
    for stream in (None, 5):
        with pytest.raises(ValueError, match="current device"):
            L._stream_on(stream, other)


@pytest.mark.parametrize("bits", [11, 8])
@pytest.mark.parametrize("M,K,group", [(300, 8192, 32), (77, 9001, 128), (130, 16384, 64)])
def test_a_unit_left_out_shows(M, K, group, bits):
    """The exact comparison of long sums (whole x, power-of-two scales) is sharp: with 128 columns left out of the
    definition almost every rounded output differs, in both 16-bit types, and so does the norm bound's error."""
    import numpy as np

    from oracle import serving as sv
    rng = np.random.default_rng(M)
    codes = rng.integers(0, 256, (M, (K + 1) // 2)).astype(np.uint8)
    c, s = sv.quant_weights(codes, 2.0 ** rng.integers(-2, 2, (M, -(-K // group))), None, K, group)
    x = rng.integers(-2, 3, (5, K)).astype(np.float64)
    whole = x @ (c * s).T
    for u in (0, K // 256, (K - 1) // 128):
        part = x.copy()
        part[:, 128 * u:128 * (u + 1)] = 0
        part = part @ (c * s).T

        def rounded(v):
            f, e = np.frexp(v)
            return np.ldexp(np.rint(f * 2.0 ** bits), e - bits)

        assert (rounded(part) != rounded(whole)).mean() > (0.9 if 128 * (u + 1) <= K else 0.5)
        assert np.linalg.norm(part - whole) > 4 * 2.0 ** -bits * np.linalg.norm(whole)
