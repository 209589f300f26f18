"""The widest tables under which pa_decode_accumulate counts a context's tokens in 32 bits."""
import pytest

from paged_kv_cache_76_gb300 import _lib


@pytest.mark.parametrize("bs", [4, 8, 16, 32])
def test_widest_table(bs):
    try:
        lib = _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
        lib = _lib.lib()
    most = (2 ** 31 - 1 - 4096) // bs
    for split in (0, 64):
        assert lib.pa_decode_accumulate_split_tokens(1, 4, 1, most, bs, split) > 0
        assert lib.pa_decode_accumulate_split_tokens(1, 4, 1, most + 1, bs, split) == _lib.PA_ERR_INVALID
        assert lib.pa_decode_accumulate_workspace_size(1, 4, 1, 64, most + 1, bs, split) == 0
