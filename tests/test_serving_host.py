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
