"""Refusals of the 4-bit cache's calls, fork_blocks and copy_pages before
anything is launched: the binding's checks on CPU tensors, and the C calls' own
on sizes and pointers; and the row-by-row form of fork_blocks by hand."""
import pytest
import torch

import fork_ref
import kv4_ref
from paged_kv_cache_76_gb300 import _lib, ops

BF = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    try:
        return _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
        return _lib.lib()


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


def kv(nb=4, bs=16, hkv=2, d=128):
    return [ops.kv4_cache(nb, bs, hkv, d, device="cpu") for _ in range(2)]


def refuser(f, good):
    def refused(error, **kw):
        with pytest.raises(error):
            f(**{**good, **kw})
    refused(ValueError)  # CPU tensors (all checks passed)
    return refused


def test_cache_shapes():
    assert kv()[0].shape == (4, 2, 16 * 72) and kv(bs=4, d=64)[0].shape == (4, 2, 144)
    for bad in (dict(bs=12), dict(d=96), dict(bs=64)):
        with pytest.raises(ValueError):
            kv(**bad)


def test_write_and_read_bindings(lib):
    kc, vc = kv()
    k = torch.zeros(5, 2, 128, dtype=BF)
    refused = refuser(ops.quantize_and_cache, dict(k=k, v=k, slot_mapping=i32(5), k_cache=kc, v_cache=vc))
    refused(TypeError, k=k.float(), v=k.float())
    refused(TypeError, v=k.half())
    refused(ValueError, v=k[:4])
    refused(ValueError, k=k[0], v=k[0])
    refused(ValueError, k=torch.zeros(5, 3, 128, dtype=BF), v=torch.zeros(5, 3, 128, dtype=BF))
    refused(ValueError, k=torch.zeros(5, 2, 96, dtype=BF), v=torch.zeros(5, 2, 96, dtype=BF))
    refused(ValueError, k=torch.zeros(5, 2, 256, dtype=BF)[..., :128])
    refused(ValueError, k=torch.zeros(1, 2, 128, dtype=BF).expand(5, 2, 128))
    refused(ValueError, slot_mapping=i32(4))
    refused(TypeError, slot_mapping=torch.zeros(5, dtype=torch.int64))
    refused(ValueError, k_cache=kc.view(torch.int8))
    refused(ValueError, v_cache=vc[:3])
    refused(ValueError, k_cache=kc[..., :100], v_cache=vc[..., :100])
    refused = refuser(ops.dequantize_kv4, dict(k_cache=kc, v_cache=vc, slots=i32(3), head_dim=128))
    refused(ValueError, head_dim=96)
    refused(ValueError, head_dim=0)
    refused(TypeError, dtype=torch.float32)
    refused(ValueError, slots=i32(3, 1))


def test_attention_bindings(lib):
    kc, vc = kv()
    q = torch.zeros(2, 8, 128, dtype=BF)
    refused = refuser(ops.decode_kv4, dict(q=q, k_cache=kc, v_cache=vc, block_tables=i32(2, 4), context_lens=i32(2),
                                           scale=0.1))
    refused(ValueError, q=q[0])
    refused(TypeError, q=q.float())
    refused(ValueError, q=torch.zeros(2, 8, 96, dtype=BF))
    refused(ValueError, block_tables=i32(3, 4))
    refused(ValueError, context_lens=i32(3))
    refused(ValueError, out=torch.zeros(2, 8, 64, dtype=BF))
    refused(ValueError, out=torch.zeros(2, 8, 128))
    refused = refuser(ops.chunked_prefill_kv4, dict(
        q=q, q_start=i32(3), context_lens=i32(2), k_cache=kc, v_cache=vc, block_tables=i32(2, 4), scale=0.1, max_q_len=1))
    refused(ValueError, q=q[None])
    refused(TypeError, q=q.float())
    refused(ValueError, q_start=i32(2))
    refused(ValueError, block_tables=i32(2))
    refused(ValueError, out=torch.zeros(3, 8, 128, dtype=BF))


def test_fork_and_copy_bindings(lib):
    refused = refuser(ops.fork_blocks, dict(block_tables=i32(2, 4), context_lens=i32(2), parents=i32(3), num_blocks=8,
                                            block_size=4))
    refused(ValueError, context_lens=i32(3))
    refused(TypeError, parents=torch.zeros(3, dtype=torch.int64))
    refused(ValueError, grow=i32(3))
    refused(ValueError, grow=i32(2), max_grow=1)
    refused(ValueError, grow=2, max_grow=1)
    refused(ValueError, grow=-1)
    refused(ValueError, pinned=torch.zeros(7, dtype=torch.bool))
    refused(ValueError, pinned=i32(8))
    refused(ValueError, max_blocks=0)
    a, b = torch.zeros(6, 4, 2, 64, dtype=BF), torch.zeros(6, 2, 144, dtype=torch.uint8)
    refused = refuser(ops.copy_pages, dict(caches=[a, a], pairs=i32(2, 2)))
    refused(ValueError, caches=[a, b])
    refused(ValueError, caches=[a, a[:5]])
    refused(ValueError, caches=[b[..., :100].contiguous()])
    refused(ValueError, pairs=i32(4))


def test_c_calls_check_before_they_launch(lib):
    inv, ws = _lib.PA_ERR_INVALID, _lib.PA_ERR_WORKSPACE
    P = 16
    q = lambda **k: lib.pa_quantize_and_cache(*{**dict(k=P, v=P, ks=256, vs=256, sl=P, T=3, kc=P, vc=P, nb=4, bs=16,  # noqa: E731
                                                       h=2, d=128, dt=1, st=None), **k}.values())
    assert q(T=0) == _lib.PA_OK and q(T=-1) == inv
    for bad in (dict(k=None), dict(sl=None), dict(k=24), dict(kc=8), dict(ks=255), dict(ks=252), dict(vs=128),
                dict(bs=12), dict(d=96), dict(h=0), dict(nb=0), dict(nb=2 ** 31 - 1), dict(ks=2 ** 62)):
        assert q(**bad) == inv, bad
    assert q(dt=2) == _lib.PA_ERR_DTYPE
    r = lambda **k: lib.pa_dequantize_kv4(*{**dict(kc=P, vc=P, sl=P, T=3, nb=4, bs=16, h=2, d=128, k=P, v=P, dt=0,  # noqa: E731
                                                   st=None), **k}.values())
    assert r(T=0) == _lib.PA_OK
    for bad in (dict(k=None), dict(v=8), dict(T=-1), dict(d=80)):
        assert r(**bad) == inv, bad
    d = lambda **k: lib.pa_decode_kv4(*{**dict(q=P, kc=P, vc=P, tab=P, mb=64, lens=P, B=2, ql=1, hq=8, h=2, d=128, bs=16,  # noqa: E731
                                               nb=99, sc=0.1, sp=32, ws=P, wb=1 << 30, out=P, dt=1, st=None), **k}.values())
    assert d(B=0) == _lib.PA_OK
    for bad in (dict(q=None), dict(out=8), dict(tab=None), dict(B=-1), dict(B=65536), dict(ql=0), dict(ql=9), dict(hq=9),
                dict(hq=34, h=2), dict(sp=31), dict(sp=48), dict(sp=1 << 20), dict(sc=float("nan")),
                dict(sc=float("inf")), dict(mb=0), dict(mb=2 ** 31 - 1)):
        assert d(**bad) == inv, bad
    assert d(wb=100) == ws and d(ws=None) == ws and d(ws=8) == ws
    assert lib.pa_decode_kv4_workspace_size(2, 1, 8, 2, 128, 64, 16, 32) > 2 * 8 * 32 * 128 * 4
    assert lib.pa_decode_kv4_workspace_size(2, 1, 8, 2, 128, 64, 16, 128) == 0  # eight partitions join without
    assert lib.pa_decode_kv4_workspace_size(2, 33, 8, 2, 128, 64, 16, 128) == 0
    assert lib.pa_decode_kv4_split_tokens(2, 1, 8, 2, 64, 16, 96) == 96
    assert lib.pa_decode_kv4_split_tokens(2, 1, 8, 2, 64, 16, 0) % 32 == 0
    p = lambda **k: lib.pa_chunked_prefill_kv4(*{**dict(  # noqa: E731
        q=P, qs=P, lens=P, kc=P, vc=P, tab=P, mb=64, R=2, T=20, mq=16, hq=8, h=2, d=128, bs=16, nb=99, sc=0.1, sp=64,
        ws=P, wb=1 << 30, out=P, dt=1, st=None), **k}.values())
    assert p(R=0) == _lib.PA_OK and p(T=0) == _lib.PA_OK
    for bad in (dict(q=None), dict(qs=None), dict(q=8), dict(R=65536), dict(T=-1), dict(mq=0), dict(hq=34, h=2),
                dict(sp=63), dict(sp=-64), dict(sc=0.0), dict(sc=1e-40), dict(sc=float("inf")), dict(sc=3e38),
                dict(mq=2 ** 31 - 1)):
        assert p(**bad) == inv, bad
    assert p(wb=16) == ws
    f = lambda **k: lib.pa_fork_blocks(*{**dict(  # noqa: E731
        tab=1 << 20, mb=8, lens=2 << 20, B=4, par=3 << 20, R=4, gr=None, mg=1, pin=None, nb=100, bs=16, to=4 << 20, mo=8,
        lo=5 << 20, pr=6 << 20, sl=7 << 20, nf=8 << 20, ws=9 << 20, wb=1 << 20, st=None), **k}.values())
    for bad in (dict(tab=None), dict(par=None), dict(to=None), dict(sl=None), dict(nf=None), dict(bs=12), dict(nb=0),
                dict(nb=2 ** 30), dict(B=65536), dict(R=65536), dict(mg=-1), dict(mo=0), dict(mb=0), dict(mb=2 ** 30),
                dict(to=1 << 20), dict(to=(1 << 20) + 64), dict(lo=2 << 20), dict(lo=(3 << 20) + 4), dict(pr=4 << 20),
                dict(sl=8 << 20), dict(nf=9 << 20), dict(mg=129), dict(gr=5 << 20, mg=2), dict(pin=7 << 20)):
        assert f(**bad) == inv, bad
    assert f(ws=None) == ws and f(wb=64) == ws and f(ws=(9 << 20) + 8) == ws
    import ctypes
    arr = (ctypes.c_void_p * 2)(16, 8)
    assert lib.pa_copy_pages(arr, 2, P, 1, 4, 64, None) == inv          # a cache that is not aligned
    assert lib.pa_copy_pages(arr, 1, P, 0, 4, 64, None) == _lib.PA_OK
    assert lib.pa_copy_pages(arr, 0, P, 1, 4, 64, None) == _lib.PA_OK
    for bad in ((arr, 1, None, 1, 4, 64), (None, 1, P, 1, 4, 64), (arr, 1, P, -1, 4, 64), (arr, 1, P, 1, 0, 64),
                (arr, 1, P, 1, 4, 24), (arr, 1, P, 1, 4, 0)):
        assert lib.pa_copy_pages(*bad, None) == inv, bad


def test_the_forms_the_gpu_is_compared_with():
    # two rows go on inside block 9; row 2 is left: 3 and 7 come back, 0 and 1 are free
    t, n, p, s, free = fork_ref.fork([[4, 9, -1], [4, 9, -1], [7, 3, -1]], [6, 6, 7], [0, 1], [1, 1], 10, 4, 3, 1)
    assert t == [[4, 9, -1], [4, 0, -1]] and n == [7, 7] and p == [[-1, -1], [9, 0]] and s == [[38], [2]] and free == 7
    # 5 / 6 is nearest to 0.8125; 0.3125 / 0.8125 = 0.38.. to 0.5; 2.03125 (2.5 of the scale) is a tie: level 2
    x = torch.zeros(16, dtype=torch.float64)
    x[0], x[1], x[2], x[3] = 5.0, 0.3125, 2.03125, -0.203125
    v, byte = kv4_ref.quantized(x)
    assert float(kv4_ref.scale_values()[byte]) == 0.8125
    assert v[:4].tolist() == [4.875, 0.40625, 1.625, 0.0]
    page = torch.zeros(1, 1, 4 * 36, dtype=torch.uint8)
    page[0, 0, 32] = 0x7F                      # token 1, elements 0 and 1: -6 and 6
    page[0, 0, 4 * 32 + 4] = 0x78              # its first scale: 1
    page[0, 0, 4 * 32 + 5] = 0xFF
    got = kv4_ref.numbers(page, 4, 64)
    assert got[0, 1, 0, :3].tolist() == [-6.0, 6.0, 0.0] and bool(got[0, 1, 0, 16:32].isnan().all())
