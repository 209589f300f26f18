"""Refusals of norm_rope_and_cache, verify_tree, decode_accumulate,
evict_select and compact_kv before anything is launched: the binding's checks
on CPU tensors, and the C calls' own on sizes and pointers."""
import pytest
import torch

from paged_kv_cache_76_gb300 import _lib, ops


@pytest.fixture(scope="module")
def lib():
    try:
        return _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
        return _lib.lib()


def kv(nb=4, bs=16, hkv=2, d=128, dt=torch.bfloat16):
    return torch.zeros(nb, bs, hkv, d, dtype=dt), torch.zeros(nb, bs, hkv, d, dtype=dt)


def i32(*shape):
    return torch.zeros(*shape, dtype=torch.int32)


BF = torch.bfloat16


def test_norm_rope_binding():
    kc, vc = kv()
    good = dict(q=torch.zeros(5, 8, 128, dtype=BF), k=torch.zeros(5, 2, 128, dtype=BF),
                v=torch.zeros(5, 2, 128, dtype=BF), positions=i32(5), cos_sin=torch.zeros(100, 64),
                slot_mapping=i32(5), k_cache=kc, v_cache=vc)

    def refused(error, **kw):
        with pytest.raises(error):
            ops.norm_rope_and_cache(**{**good, **kw})

    refused(ValueError)                                                    # CPU tensors (all checks passed)
    refused(TypeError, q=good["q"].half())
    refused(ValueError, q=torch.zeros(5, 8, 64, dtype=BF))
    refused(ValueError, k=torch.zeros(4, 2, 128, dtype=BF))
    refused(ValueError, v=torch.zeros(5, 3, 128, dtype=BF))
    refused(ValueError, q=torch.zeros(5, 8, 256, dtype=BF)[..., :128])     # heads not contiguous
    refused(ValueError, q=torch.zeros(5, 8 * 128 + 4, dtype=BF)[:, :1024].unflatten(1, (8, 128)))  # stride not of 8
    refused(ValueError, q=torch.zeros(1, 8, 128, dtype=BF).expand(5, 8, 128))                      # tokens overlap
    refused(ValueError, positions=i32(4))
    refused(ValueError, positions=i32(4, 5))                               # four axes
    refused(ValueError, positions=i32(2, 5))                               # sections missing
    refused(ValueError, positions=i32(2, 5), sections=(16, 15))            # not rot_dim / 2
    refused(ValueError, positions=i32(2, 5), sections=(40, -8))
    refused(ValueError, cos_sin=torch.zeros(100, 64, dtype=torch.float64))
    refused(ValueError, q_weight=torch.zeros(64, dtype=BF))
    refused(ValueError, k_weight=torch.zeros(128))
    refused(ValueError, slot_mapping=i32(6))
    refused(ValueError, out=torch.zeros(5, 8, 128))


def test_verify_tree_binding():
    kc, vc = kv()
    good = dict(q=torch.zeros(5, 8, 128, dtype=BF), q_start=i32(3), tree_mask=torch.zeros(5, dtype=torch.int64),
                context_lens=i32(2), k_cache=kc, v_cache=vc, block_tables=i32(2, 4), scale=0.1, max_q_len=3)

    def refused(error, **kw):
        with pytest.raises(error):
            ops.verify_tree(**{**good, **kw})

    refused(TypeError, q=good["q"].half())
    refused(ValueError, q=good["q"][0])
    refused(ValueError, q_start=i32(2))
    refused(TypeError, tree_mask=i32(5))
    refused(ValueError, tree_mask=torch.zeros(4, dtype=torch.int64))
    refused(ValueError, block_tables=i32(3, 4))
    refused(ValueError, out=torch.zeros(4, 8, 128, dtype=BF))
    with pytest.raises(ValueError):
        ops.tree_mask([-1, 1])                                             # its own parent
    with pytest.raises(ValueError):
        ops.tree_mask([-1] * 65)
    assert ops.tree_mask([-1, 0, 0, 2, -1]).tolist() == [1, 3, 5, 13, 16]
    assert ops.tree_mask([i - 1 for i in range(64)]).tolist()[-1] == -1    # bit 63 is the sign


def test_eviction_bindings():
    kc, vc = kv()
    q, s = torch.zeros(3, 8, 128, dtype=BF), torch.zeros(3, 2, 64)
    with pytest.raises(ValueError):
        ops.decode_accumulate(q, kc, vc, i32(3, 4), i32(3), 0.1, s[:2])                 # fewer rows than requests
    with pytest.raises(ValueError):
        ops.decode_accumulate(q, kc, vc, i32(3, 4), i32(3), 0.1, s.double())
    with pytest.raises(ValueError):
        ops.decode_accumulate(q, kc, vc, i32(3, 4), i32(3), 0.1, torch.zeros(3, 4, 64))
    with pytest.raises(ValueError):
        ops.decode_accumulate(q, kc, vc, i32(3, 4), i32(3), 0.1, s, scores_out=torch.zeros(3, 2, 65))
    with pytest.raises(ValueError):
        ops.decode_accumulate(q, kc, vc, i32(3, 4), i32(3), 0.1, s, score_rows=i32(2))
    for sink, heavy, recent in ((0, 0, 0), (-1, 4, 4), (1, -2, 4)):
        with pytest.raises(ValueError):
            ops.evict_select(s, i32(3), sink, heavy, recent)
    with pytest.raises(ValueError):
        ops.evict_select(s, i32(3), 1, 2, 3, keep=i32(3, 2, 7))
    with pytest.raises(ValueError):
        ops.evict_select(s, i32(3), 1, 2, 3, keep_lens=i32(2))
    with pytest.raises(ValueError):
        ops.compact_kv(kc, vc, i32(3, 4), i32(3), i32(3, 3, 5), i32(3))                 # neither 1 nor kv_heads lists
    with pytest.raises(ValueError):
        ops.compact_kv(kc, vc, i32(3, 4), i32(3), i32(3, 2, 5), i32(2))
    with pytest.raises(ValueError):
        ops.compact_kv(kc, vc, i32(3, 4), i32(3), i32(3, 2, 5), i32(3), base=i32(4))
    with pytest.raises(ValueError):
        ops.compact_kv(kc, vc, i32(3, 4), i32(3), i32(3, 2, 0), i32(3), scores=s)


def test_c_calls_check_sizes_and_pointers(lib):
    inv, ok, dt = _lib.PA_ERR_INVALID, _lib.PA_OK, _lib.PA_ERR_DTYPE
    P = 16  # a non-null, 16-byte aligned "pointer": every call below returns before it is used

    def rope(qs=1024, ks=256, eps=1e-6, axes=1, sec=None, maxp=10, rot=64, T=1, hq=8, nb=4, bs=16, hkv=2, d=128,
             dtype=1, q=P, out=P, cos=P):
        return lib.pa_norm_rope_and_cache(q, P, P, qs, ks, ks, None, None, eps, P, axes, sec, cos, maxp, rot, 0, P, T,
                                          hq, out, P, P, nb, bs, hkv, d, dtype, None)

    assert rope(dtype=7) == dt
    for kw in (dict(d=96), dict(bs=12), dict(rot=8), dict(rot=40), dict(rot=144), dict(axes=0), dict(axes=4),
               dict(axes=2), dict(maxp=0), dict(T=-1), dict(hq=0), dict(qs=1016), dict(qs=1028), dict(ks=248),
               dict(eps=float("nan")), dict(eps=-1.0), dict(q=8), dict(out=None), dict(cos=4),
               dict(qs=2048, q=P, out=P)):                     # in place needs contiguous rows
        assert rope(**kw) == inv, kw
    import ctypes as C
    assert rope(axes=2, sec=(C.c_int32 * 2)(16, 15)) == inv
    assert rope(axes=3, sec=(C.c_int32 * 3)(40, -8, 0)) == inv
    assert rope(T=0, q=None) == ok

    def tree(R=1, T=4, maxq=4, hq=8, hkv=2, d=128, bs=16, nb=4, maxblk=8, split=0, ws=None, wb=0, scale=0.1, mask=P,
             dtype=1):
        return lib.pa_verify_tree(P, P, mask, P, P, P, P, maxblk, R, T, maxq, hq, hkv, d, bs, nb, scale, split, ws, wb,
                                  P, dtype, None)

    assert tree(dtype=3) == dt
    for kw in (dict(maxq=0), dict(maxq=65), dict(hq=9), dict(hq=34), dict(R=-1), dict(R=65536), dict(T=-1),
               dict(maxblk=0), dict(maxblk=1 << 28), dict(split=64), dict(split=-128), dict(mask=4), dict(mask=None),
               dict(scale=float("inf")), dict(T=1 << 30)):
        assert tree(**kw) == inv, kw
    assert tree(maxblk=64, split=128) == _lib.PA_ERR_WORKSPACE
    assert tree(R=0) == ok and tree(T=0) == ok
    assert lib.pa_verify_tree_split_tokens(64, 60, 32, 8, 256, 16, 0) == 4096       # enough units: whole contexts
    assert lib.pa_verify_tree_split_tokens(1, 60, 32, 8, 504, 16, 0) == 512         # few: twice the 240 rows
    assert lib.pa_verify_tree_split_tokens(1, 4, 8, 8, 504, 16, 0) == 512           # a unit on seven SMs in eight
    assert lib.pa_verify_tree_split_tokens(2, 4, 8, 8, 32, 16, 0) == 256            # the smallest
    assert lib.pa_verify_tree_split_tokens(1, 4, 8, 8, 504, 16, 200) == inv
    assert lib.pa_verify_tree_workspace_size(64, 640, 10, 32, 8, 128, 256, 16, 0) == 0
    assert lib.pa_verify_tree_workspace_size(1, 10, 10, 32, 8, 128, 256, 16, 512) >= 8 * 10 * 32 * 130 * 4

    def acc(R=2, hq=8, hkv=2, maxblk=8, split=0, rows=P, num_rows=2, slen=128, ws=P, wb=1 << 30, s=P, so=P):
        return lib.pa_decode_accumulate(P, P, P, P, maxblk, P, R, hq, hkv, 128, 16, 4, 0.1, split, s, rows, num_rows,
                                        slen, so, ws, wb, P, 1, None)

    for kw in (dict(R=-1), dict(hq=9), dict(hq=34), dict(maxblk=0), dict(split=24), dict(num_rows=0), dict(slen=0),
               dict(rows=None, num_rows=1), dict(s=None), dict(so=4)):
        assert acc(**kw) == inv, kw
    assert acc(ws=None) == _lib.PA_ERR_WORKSPACE and acc(wb=64) == _lib.PA_ERR_WORKSPACE
    assert acc(R=0, ws=None) == ok
    # a batch of thousands of warps keeps decode's partitions, a small one is cut finer, a huge one coarser
    assert lib.pa_decode_accumulate_split_tokens(64, 32, 8, 256, 16, 0) == 384
    assert lib.pa_decode_accumulate_split_tokens(4, 28, 4, 94, 16, 0) == 64
    assert lib.pa_decode_accumulate_split_tokens(8, 64, 8, 8192, 16, 0) == 1024
    assert lib.pa_decode_accumulate_split_tokens(4, 28, 4, 94, 16, 256) == 256
    assert lib.pa_decode_accumulate_workspace_size(4, 28, 4, 128, 94, 16, 256) >= (
        4 * 28 * 6 * 131 + 4 * 4 * 8 * 94 * 16) * 4     # the group of 7 lies in 8 columns

    def sel(rows=P, num_rows=2, hkv=2, slen=64, R=2, sink=1, heavy=2, recent=3, s=P, keep=P):
        return lib.pa_evict_select(s, rows, num_rows, hkv, slen, P, R, sink, heavy, recent, keep, P, None)

    for kw in (dict(num_rows=0), dict(hkv=0), dict(slen=0), dict(R=-1), dict(R=65536), dict(sink=-1), dict(heavy=-1),
               dict(recent=-1), dict(sink=0, heavy=0, recent=0), dict(heavy=2**31 - 1), dict(rows=None, num_rows=1),
               dict(s=None), dict(keep=None)):
        assert sel(**kw) == inv, kw
    assert sel(R=0, s=None) == ok

    def com(maxblk=8, heads=2, maxk=4, R=2, nb=4, bs=16, hkv=2, d=128, dtype=1, s=None, rows=None, num_rows=0, slen=0,
            k=P, keep=P):
        return lib.pa_compact_kv(k, P, P, maxblk, P, keep, heads, maxk, P, None, R, nb, bs, hkv, d, dtype, s, rows,
                                 num_rows, slen, None)

    assert com(dtype=9) == dt
    for kw in (dict(maxblk=0), dict(heads=3), dict(maxk=0), dict(maxk=2**31 - 1), dict(R=-1), dict(R=65536),
               dict(d=96), dict(s=P), dict(s=P, num_rows=1, slen=10), dict(s=4, num_rows=2, slen=10), dict(k=8),
               dict(keep=None)):
        assert com(**kw) == inv, kw
    assert com(R=0, keep=None) == ok


def test_select_refuses_outputs_that_lie_in_its_inputs(lib):
    """Every CTA of a row reads the lengths, rows and scores while others write the lists and their lengths."""
    S, L, R, K, N = 1 << 20, 2 << 20, 3 << 20, 4 << 20, 5 << 20   # no call below reaches the GPU: it is refused first

    def sel(s=S, lens=L, rows=R, keep=K, n=N, R=2, budget=6):
        return lib.pa_evict_select(s, rows, 2, 2, 64, lens, R, 1, budget - 4, 3, keep, n, None)

    for kw in (dict(n=L), dict(n=L + 4), dict(lens=L, n=L - 4), dict(n=R), dict(n=S + 1020), dict(keep=L),
               dict(keep=L - 80), dict(keep=R), dict(keep=S), dict(keep=S + 1008), dict(n=K), dict(n=K + 92)):
        assert sel(**kw) == _lib.PA_ERR_INVALID, kw
    assert sel(R=0, n=L) == _lib.PA_OK


def test_tree_scale_is_positive(lib):
    """Masked logits are -inf before they are scaled: a scale of zero or below would make them NaN or +inf."""
    P = 16

    def tree(scale, maxblk=8):
        return lib.pa_verify_tree(P, P, P, P, P, P, P, maxblk, 1, 4, 4, 8, 2, 128, 16, 4, scale, 128, None, 0, P, 1, None)

    for scale in (0.0, -0.0, -0.125, 1e-40, float("nan"), float("-inf")):
        assert tree(scale) == _lib.PA_ERR_INVALID, scale
    assert tree(1e-37, maxblk=64) == _lib.PA_ERR_WORKSPACE       # this far it gets with any other


def test_accumulate_refuses_scores_that_overlap_in_part(lib):
    """Each entry is read and written once, by the thread that owns it: in place or apart, not shifted."""
    P, S = 16, 1 << 20
    size = 2 * 2 * 128 * 4

    def acc(s, so, rows=None, ws=P):
        return lib.pa_decode_accumulate(P, P, P, P, 8, P, 2, 8, 2, 128, 16, 4, 0.1, 0, s, rows, 2, 128, so, ws, 64, P, 1,
                                        None)

    for so in (S + 16, S - 16, S + size - 16, S - size + 16):
        assert acc(S, so) == _lib.PA_ERR_INVALID, so
    for so in (S, S + size, S - size):                           # these get as far as the scratch's size
        assert acc(S, so) == _lib.PA_ERR_WORKSPACE, so
