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


def test_e2m1_codes_and_scales():
    """The 4-bit groups' definition: the scale's steps at 6 * 2^e, ties to the even code, what is not finite."""
    from oracle import serving as sv
    import numpy as np
    codes, byte = sv.e2m1_group([6.0, 5.0, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25, -0.25, -5.01])
    assert byte == 127 and codes.tolist() == [7, 6, 6, 4, 4, 2, 2, 0, 8, 15]
    assert sv.e2m1_group([6.01])[1] == 128 and sv.e2m1_group([3.0])[1] == 126 and sv.e2m1_group([0.0])[1] == 127
    assert sv.e2m1_group([2.0 ** -140])[1] == 1 and sv.e2m1_group([np.inf, 1.0])[1] == 255
    packed = np.array([[[0x71, 0xF0]]], dtype=np.uint8)
    assert sv.e2m1_values(packed, np.array([[[128, 0]]], dtype=np.uint8), 4).tolist() == [[[1.0, 12.0, 0.0, -12.0]]]


def cache_of(kind=None, **more):
    c = dict(k=0x1000, v=0x2000, k_scale=0x3000, v_scale=0x4000, num_pages=8, heads=2, page_size=16, head_dim=64, type=L.LSCD_E2M1)
    c.update(more)
    return L.lscd_cache_t(*c.values())


def weigh_status(cache=None, **more):
    """Status of lscd_cache_weigh for arrays that are not there."""
    a = dict(q=0x5000, q_stride=256, q_heads=4, lse=0x6000, start=0x7000, length=0x7100, table=0x7200, table_stride=4,
             table_pages=4, sequences=3, T=5, scale=0.1, causal=1, window=0, weight=0x8000, type=L.LSCD_F16)
    a.update(more)
    return L._lib.lscd_cache_weigh(ctypes.byref(cache if cache is not None else cache_of()), *a.values(), None)


def evict_status(cache=None, **more):
    a = dict(weight=0x8000, length=0x7100, table=0x7200, table_stride=4, table_pages=4, to=None, to_stride=0, to_pages=0,
             sequences=3, keep=20, recent=4, kept=0x9000)
    a.update(more)
    return L._lib.lscd_cache_evict(ctypes.byref(cache if cache is not None else cache_of()), *a.values(), None)


CACHES = [dict(k=None), dict(k_scale=None), dict(k=0x1008), dict(v_scale=0x4004), dict(num_pages=0), dict(type=7)]
LIMITS = [dict(page_size=24), dict(head_dim=40), dict(head_dim=272), dict(heads=65536), dict(num_pages=2 ** 28)]


@pytest.mark.parametrize("call", [weigh_status, evict_status])
def test_caches_are_checked(call):
    for bad in CACHES:
        assert call(cache_of(**bad)) == L.LSCD_ERROR_INVALID_VALUE, bad
    for bad in LIMITS:
        assert call(cache_of(**bad)) == L.LSCD_ERROR_NOT_SUPPORTED, bad


def test_weigh_refuses():
    for bad in (dict(q=None), dict(q=0x5008), dict(q_stride=255), dict(q_stride=128), dict(q_heads=3), dict(q_heads=0), dict(lse=None),
                dict(lse=0x6002), dict(weight=None), dict(weight=0x8004), dict(start=None), dict(length=0x7102), dict(table=None),
                dict(table_pages=0), dict(table_stride=3), dict(T=-1), dict(sequences=-1), dict(window=-1),
                dict(scale=float("nan")), dict(type=L.LSCD_E4M3)):
        assert weigh_status(**bad) == L.LSCD_ERROR_INVALID_VALUE, bad
    assert weigh_status(cache_of(type=L.LSCD_BF16, k_scale=None, v_scale=None)) == L.LSCD_ERROR_NOT_SUPPORTED
    assert weigh_status(T=2 ** 31) == L.LSCD_ERROR_NOT_SUPPORTED
    assert weigh_status(table_pages=2 ** 27, table_stride=2 ** 27) == L.LSCD_ERROR_NOT_SUPPORTED
    # 2^31 units: 16 query rows by 32 positions, a key head each
    assert weigh_status(T=2 ** 24, table_pages=2 ** 14, table_stride=2 ** 14) == L.LSCD_ERROR_NOT_SUPPORTED
    for nothing in (dict(T=0), dict(sequences=0), dict(T=0, q=None, lse=None, weight=None, table=None)):
        assert weigh_status(**nothing) == L.LSCD_SUCCESS, nothing


def test_evict_refuses():
    for bad in (dict(keep=0), dict(recent=-1), dict(recent=21), dict(sequences=-1), dict(weight=None), dict(weight=0x8008),
                dict(length=None), dict(table=0x7202), dict(table_pages=0), dict(table_stride=3), dict(kept=None), dict(kept=0x9001),
                dict(to=0xA002, to_stride=4, to_pages=4), dict(to=0xA000, to_stride=4, to_pages=1),
                dict(to=0xA000, to_stride=1, to_pages=2), dict(to=0xA000, to_stride=0, to_pages=0)):
        assert evict_status(**bad) == L.LSCD_ERROR_INVALID_VALUE, bad
    assert evict_status(table_pages=2 ** 27, table_stride=2 ** 27) == L.LSCD_ERROR_NOT_SUPPORTED
    assert evict_status(sequences=2 ** 21) == L.LSCD_ERROR_NOT_SUPPORTED
    assert evict_status(sequences=2 ** 30, cache=cache_of(heads=65535)) == L.LSCD_ERROR_NOT_SUPPORTED
    assert evict_status(sequences=0, weight=None, kept=None, table=None) == L.LSCD_SUCCESS


def test_evict_refuses_more_than_it_counts():
    """Numbers of positions past 2^30, whose loops and launches would pass 31 bits, in place and into other pages."""
    for keep in (2 ** 30 + 1, 2 ** 31 - 64, 2 ** 31 - 1):
        for more in (dict(), dict(recent=keep), dict(to=0xA000, to_stride=2 ** 27, to_pages=2 ** 27)):
            assert evict_status(sequences=1, keep=keep, **{"recent": 0, **more}) == L.LSCD_ERROR_NOT_SUPPORTED, (keep, more)
