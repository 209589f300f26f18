"""The scales that the 4-bit cache's attention takes: the kernels count scores in log2 units, and a scale that is not
finite there would make a row whose products are all zero NaN."""
import numpy as np
import pytest

from paged_kv_cache_76_gb300 import _lib

P = 16
LARGEST = float(np.finfo(np.float32).max)


@pytest.fixture(scope="module")
def lib():
    try:
        return _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
        return _lib.lib()


def decode(lib, scale):  # of an empty batch
    return lib.pa_decode_kv4(P, P, P, P, 64, P, 0, 1, 8, 2, 128, 16, 99, scale, 0, None, 0, P, 1, None)


def prefill(lib, scale):
    return lib.pa_chunked_prefill_kv4(P, P, P, P, P, P, 64, 0, 0, 0, 8, 2, 128, 16, 99, scale, 0, None, 0, P, 1, None)


@pytest.mark.parametrize("call", [decode, prefill])
def test_scales(lib, call):
    for scale in (0.09, -0.09, 1e-30, LARGEST * 0.69, -LARGEST * 0.69):
        assert call(lib, scale) == _lib.PA_OK, scale
    for scale in (LARGEST, -LARGEST, LARGEST * 0.7, float("inf"), float("nan")):
        assert call(lib, scale) == _lib.PA_ERR_INVALID, scale
    for scale in (0.0, 1e-40):  # prefill masks before it scales
        assert call(lib, scale) == (_lib.PA_OK if call is decode else _lib.PA_ERR_INVALID)
