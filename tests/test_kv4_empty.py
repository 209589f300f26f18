"""Empty batches of the 4-bit cache's calls are no work, whatever they leave the
library to choose: a step without a prompt, requests without a query."""
import pytest
import torch

from paged_kv_cache_76_gb300 import _lib, ops

P = 16  # a pointer that nothing reads


@pytest.fixture(scope="module")
def lib():
    try:
        return _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
        return _lib.lib()


def prefill(lib, reqs, total_q, max_q, split, width=64):
    return lib.pa_chunked_prefill_kv4(P, P, P, P, P, P, width, reqs, total_q, max_q, 8, 2, 128, 16, 99, 0.1, split, None, 0,
                                      P, 1, None)


@pytest.mark.parametrize("split", [0, 64])
@pytest.mark.parametrize("reqs,total_q,max_q", [(0, 0, 0), (0, 0, 16), (0, 20, 16), (0, 20, 0), (3, 0, 0), (3, 0, 16)])
def test_prefill_of_nothing(lib, reqs, total_q, max_q, split):
    for width in (1, 64, 8192, 2 ** 27 - 300):
        assert prefill(lib, reqs, total_q, max_q, split, width) == _lib.PA_OK
    assert prefill(lib, reqs, total_q, max_q, 63) == _lib.PA_ERR_INVALID
    for width in (1, 64, 8192):
        cap = width * 16
        got = lib.pa_chunked_prefill_kv4_split_tokens(reqs, max_q, 8, 2, width, 16, split)
        assert 64 <= got <= max(cap, 64) and got % 64 == 0
    if split == 0 and (reqs == 0 or max_q == 0):
        assert lib.pa_chunked_prefill_kv4_workspace_size(reqs, total_q, max_q, 8, 2, 128, 64, 16, 0) == 0


def test_chunks_without_room_for_their_queries(lib):
    assert prefill(lib, 3, 20, 0, 0) == _lib.PA_ERR_INVALID
    assert prefill(lib, 3, 0, -1, 0) == _lib.PA_ERR_INVALID
    assert prefill(lib, 0, 0, -1, 0) == _lib.PA_ERR_INVALID


def test_decode_of_nothing(lib):
    for split in (0, 64):
        assert lib.pa_decode_kv4(P, P, P, P, 64, P, 0, 1, 8, 2, 128, 16, 99, 0.1, split, None, 0, P, 1, None) == _lib.PA_OK
        assert lib.pa_decode_kv4_split_tokens(0, 1, 8, 2, 64, 16, split) > 0


@pytest.mark.gpu
@pytest.mark.parametrize("recorded", [False, True])
@pytest.mark.parametrize("reqs,max_q", [(0, 0), (0, 5), (2, 0), (2, 5)])
def test_empty_steps(lib, recorded, reqs, max_q):
    def i32(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device="cuda")
    kc, vc = (ops.kv4_cache(9, 16, 2, 128) for _ in range(2))
    q = torch.zeros(0, 8, 128, dtype=torch.bfloat16, device="cuda")

    def step():
        out = ops.chunked_prefill_kv4(q, i32(reqs + 1), i32(reqs), kc, vc, i32(reqs, 70), 0.1, max_q)
        assert out.shape == q.shape
        if reqs == 0:
            assert ops.decode_kv4(q, kc, vc, i32(0, 70), i32(0), 0.1).shape == q.shape
        ops.quantize_and_cache(q[:, :2], q[:, :2], i32(0), kc, vc)
        assert ops.dequantize_kv4(kc, vc, i32(0), 128)[1].shape == (0, 2, 128)
    if recorded:
        with ops.recording() as rec:
            step()
        rec()
    else:
        step()
    assert ops.get_device_error() == 0
