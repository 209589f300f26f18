"""The two ways from tensors to the C calls (the extension of csrc/marshal.cpp
and ctypes): the short one takes regular calls only and gives the same bits,
everything else goes the long way and is refused there in the same words."""
import numpy as np
import pytest
import torch

from paged_kv_cache_76_gb300 import ops

BF = torch.bfloat16
HQ, HKV, D, BS = 8, 2, 128, 16


def calls(device, dtype=BF):
    """name -> (function of ops, keyword arguments) of a small regular call."""
    g = torch.Generator().manual_seed(5)

    def x(*shape, dt=dtype):
        return torch.randn(*shape, generator=g).to(dt).to(device)

    def i32(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device=device)

    kc, vc = x(12, BS, HKV, D), x(12, BS, HKV, D)
    tables, lens = i32([[3, 1, 4, 0], [5, 9, 2, 6]]), i32([50, 33])
    qkv = x(5, (HQ + 2 * HKV) * D)
    q, k, v = (t.unflatten(1, (-1, D)) for t in qkv.split([HQ * D, HKV * D, HKV * D], 1))
    scores = x(3, HKV, 64, dt=torch.float32).abs()
    return {
        "norm_rope": (ops.norm_rope_and_cache, dict(
            q=q, k=k, v=v, positions=i32([[1, 2, 3, 4, 9]] * 2), cos_sin=ops.rope_table(32, 64, device=device),
            slot_mapping=i32([160, -1, 170, 171, 191]), k_cache=kc, v_cache=vc, q_weight=x(D), k_weight=x(D), eps=1e-5,
            sections=(20, 12), interleaved=True)),
        "tree": (ops.verify_tree, dict(
            q=x(7, HQ, D), q_start=i32([0, 4, 7]),
            tree_mask=torch.cat([ops.tree_mask([-1, 0, 0, 1]), ops.tree_mask([-1, 0, 1])]).to(device), context_lens=lens,
            k_cache=kc, v_cache=vc, block_tables=tables, scale=0.09, max_q_len=4)),
        "accumulate": (ops.decode_accumulate, dict(
            q=x(2, HQ, D), k_cache=kc, v_cache=vc, block_tables=tables, context_lens=lens, scale=0.09, scores=scores,
            score_rows=i32([2, 0]))),
        "select": (ops.evict_select, dict(scores=scores, context_lens=lens, sink=2, heavy=9, recent=5,
                                          score_rows=i32([2, 0]))),
        "compact": (ops.compact_kv, dict(
            k_cache=kc, v_cache=vc, block_tables=tables, context_lens=lens,
            keep=i32([[[0, 3, 7, 20], [1, 2, 3, 30]], [[0, 1, 2, 4], [5, 6, 7, 8]]]), keep_lens=i32([4, 3]),
            base=i32([2, 0]), scores=scores, score_rows=i32([2, 0]))),
    }


NAMES = ["norm_rope", "tree", "accumulate", "select", "compact"]


def flat(r):
    return [] if r is None else [r] if isinstance(r, torch.Tensor) else list(r)


def run(name, device="cuda", edit=None):
    """The call's outputs, and every argument tensor as it left them."""
    f, kw = calls(device)[name]
    kw.update(edit(kw) if edit else {})
    out = flat(f(**kw))
    return [t.clone() for t in out + [t for t in kw.values() if isinstance(t, torch.Tensor)]]


@pytest.fixture
def taken(monkeypatch):
    """How many calls the short way took (None: refused to) since the test began."""
    from paged_kv_cache_76_gb300 import _lib, build
    try:
        _lib.lib()
    except _lib.LibraryMissing:
        build.build()
    if not ops._load_marshal():
        pytest.skip("the extension is not built here")
    real, seen = ops._marshal, []

    class Watch:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(real, name)(*a)
                seen.append(r is not None)
                return r
            return call

    monkeypatch.setattr(ops, "_marshal", Watch())
    return seen


@pytest.mark.parametrize("name", NAMES)
def test_what_is_on_the_host_is_left_to_the_long_way(name, taken):
    f, kw = calls("cpu")[name]
    with pytest.raises(ValueError):
        f(**kw)
    assert taken == [False]
    for key in kw:                      # no argument is taken unseen
        if key in ("q_weight", "k_weight", "score_rows", "base", "sections", "scores") and name != "select":
            continue                    # may be None
        with pytest.raises((ValueError, TypeError, AttributeError)):
            f(**{**kw, key: None})
    assert not any(taken)


@pytest.mark.parametrize("name", NAMES)
def test_tensors_that_are_not_plain_are_left_to_the_long_way(name, taken):
    """Sparse and meta tensors, which have no storage to point at, and objects that are none."""
    f, kw = calls("cpu")[name]
    for key, t in kw.items():
        if not isinstance(t, torch.Tensor):
            continue
        for w in (t.to_sparse(), t.to("meta"), t.cpu().numpy() if t.dtype != BF else [1], object()):
            with pytest.raises((ValueError, TypeError, AttributeError, RuntimeError, NotImplementedError)):
                f(**{**kw, key: w})
    assert not any(taken)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_both_ways_give_the_same_bits(name, taken, monkeypatch):
    short = run(name)
    assert taken == [True]
    monkeypatch.setattr(ops, "_marshal", False)
    long = run(name)
    assert len(short) == len(long) and all(torch.equal(a, b) for a, b in zip(short, long))
    assert ops.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name,edit", [
    ("tree", lambda kw: dict(max_q_len=np.int64(4))),
    ("tree", lambda kw: dict(workspace=torch.empty(1 << 20, dtype=torch.uint8, device="cuda"))),
    ("norm_rope", lambda kw: dict(eps=np.float32(1e-5))),
    ("norm_rope", lambda kw: dict(interleaved=1)),
    ("norm_rope", lambda kw: dict(stream=torch.cuda.current_stream())),
    ("select", lambda kw: dict(heavy=np.int32(9))),
    ("accumulate", lambda kw: dict(scale=np.float32(0.09))),
])
def test_rare_forms_give_the_same_too(name, edit, taken):
    want, got = run(name), run(name, edit=edit)
    assert not any(taken[1:])
    for a, b in zip(want, got):
        assert torch.equal(a, b)


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_given_outputs_and_repeats(name, taken):
    f, kw = calls("cuda")[name]
    if name in ("norm_rope", "tree", "accumulate"):
        out = torch.zeros(kw["q"].shape, dtype=BF, device="cuda")
        got = f(**kw, out=out)
        assert (got if name != "accumulate" else got[0]) is out and taken == [True]
        assert bool((out != 0).any())
    if name == "accumulate":
        to = torch.zeros_like(kw["scores"])
        got = f(**kw, scores_out=to)
        assert got[1] is to and f(**kw)[1] is kw["scores"] and taken == [True] * 3


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_refusals_are_the_long_ways(name, taken):
    """Tensors of another type, shape, layout or place, one argument at a time: refused, and nothing launched."""
    from paged_kv_cache_76_gb300 import PAError
    f, kw = calls("cuda")[name]
    before = ops.launch_count()
    for key, t in kw.items():
        if not isinstance(t, torch.Tensor):
            continue
        wrong = [t.cpu(), t.to(torch.float64 if t.is_floating_point() else torch.int16)]
        if not (name == "norm_rope" and key == "cos_sin"):       # any number of positions
            wrong.append(torch.cat([t, t]))
        if name == "norm_rope" and key in ("k_cache", "v_cache", "positions") or key in ("k_cache", "v_cache"):
            wrong = wrong[:2]
        if key in ("scores",):
            wrong = wrong[:2]                                    # more rows than requests are fine
        wrong.append(t.to_sparse())
        if not (name == "norm_rope" and key in ("q", "k", "v")):
            wrong.append(torch.stack([t, t], -1)[..., 0])        # not contiguous
        for w in wrong:
            with pytest.raises((ValueError, TypeError, RuntimeError, NotImplementedError, PAError)):
                f(**{**kw, key: w})
    assert not any(taken) and ops.launch_count() == before
