"""The two ways from tensors to the calls of the 4-bit cache, fork_blocks and
copy_pages (the extension of csrc/marshal.cpp and ctypes): the short one takes
regular calls only and gives the same bits, everything else goes the long way
and is refused there."""
import numpy as np
import pytest
import torch

from paged_kv_cache_76_gb300 import ops

BF = torch.bfloat16
HQ, HKV, D, BS, NB = 8, 2, 128, 16, 12


def calls(device, dtype=BF):
    """name -> (function of ops, keyword arguments) of a small regular call."""
    g = torch.Generator().manual_seed(5)

    def x(*shape):
        return torch.randn(*shape, generator=g).to(dtype).to(device)

    def i32(a):
        return torch.tensor(np.asarray(a), dtype=torch.int32, device=device)

    kc, vc = (torch.randint(0, 0x70, (NB, HKV, BS * D * 9 // 16), generator=g).to(torch.uint8).to(device)
              for _ in range(2))
    tables, lens = i32([[3, 1, 4, 0], [5, 9, 2, 6]]), i32([50, 33])
    kv = x(5, 2 * HKV * D)
    k, v = (t.unflatten(1, (HKV, D)) for t in kv.chunk(2, 1))
    caches = dict(k_cache=kc, v_cache=vc)
    return {
        "quantize": (ops.quantize_and_cache, dict(k=k, v=v, slot_mapping=i32([160, -1, 170, 171, 191]), **caches)),
        "dequantize": (ops.dequantize_kv4, dict(**caches, slots=i32([4, -1, 100]), head_dim=D, dtype=dtype)),
        "decode": (ops.decode_kv4, dict(q=x(2, HQ, D), **caches, block_tables=tables, context_lens=lens, scale=0.09)),
        "verify": (ops.decode_kv4, dict(q=x(2, 3, HQ, D), **caches, block_tables=tables, context_lens=lens, scale=0.09,
                                        split_tokens=32)),
        "prefill": (ops.chunked_prefill_kv4, dict(
            q=x(7, HQ, D), q_start=i32([0, 4, 7]), context_lens=lens, **caches, block_tables=tables, scale=0.09,
            max_q_len=4)),
        "fork": (ops.fork_blocks, dict(
            block_tables=tables, context_lens=lens, parents=i32([0, 0, 1, -1]), num_blocks=NB, block_size=BS,
            grow=i32([1, 3, 0, 2]), max_grow=3, pinned=torch.zeros(NB, dtype=torch.bool, device=device), max_blocks=5)),
        "copy": (ops.copy_pages, dict(caches=[kc, vc], pairs=i32([[3, 11], [-1, -1], [5, 10]]))),
    }


NAMES = ["quantize", "dequantize", "decode", "verify", "prefill", "fork", "copy"]
OPTIONAL = ("pinned", "max_blocks", "max_grow", "grow", "head_dim", "dtype", "split_tokens", "num_blocks", "block_size")


def flat(r):
    return [] if r is None else [r] if isinstance(r, torch.Tensor) else list(r)


def tensors(kw):
    return [t for a in kw.values() for t in (a if isinstance(a, list) else [a]) if isinstance(t, torch.Tensor)]


def run(name, device="cuda", edit=None):
    """The call's outputs, and every argument tensor as it left them."""
    f, kw = calls(device)[name]
    kw.update(edit(kw) if edit else {})
    out = flat(f(**kw))
    return [t.clone() for t in out + tensors(kw)]


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
def test_what_is_on_the_host_or_no_tensor_is_left_to_the_long_way(name, taken):
    f, kw = calls("cpu")[name]
    with pytest.raises(ValueError):
        f(**kw)
    assert taken == [False]
    for key, t in kw.items():
        if key in OPTIONAL:
            continue
        with pytest.raises((ValueError, TypeError, AttributeError)):
            f(**{**kw, key: None})
        if isinstance(t, torch.Tensor):
            for w in (t.to_sparse(), t.to("meta"), object()):
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
    assert len(short) == len(long)
    assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(short, long))
    assert ops.get_device_error() == 0


@pytest.mark.gpu
@pytest.mark.parametrize("name", NAMES)
def test_irregular_calls_are_left_to_the_long_way(name, taken):
    f, kw = calls("cuda")[name]
    edits = {
        "quantize": [dict(k=kw.get("k", None) if name != "quantize" else kw["k"].float()), dict(v_cache=None)],
        "dequantize": [dict(head_dim=96), dict(slots=None), dict(dtype=torch.float32)],
        "decode": [dict(q=0), dict(split_tokens=2.5), dict(scale="x"), dict(context_lens=None)],
        "verify": [dict(block_tables=None), dict(out=kw.get("k_cache"))],
        "prefill": [dict(max_q_len=None), dict(q_start=kw.get("context_lens")), dict(scale=0.0)],
        "fork": [dict(max_grow=None), dict(pinned=kw.get("parents")), dict(block_size=12), dict(max_blocks=0)],
        "copy": [dict(pairs=kw.get("pairs", None) if name != "copy" else kw["pairs"][:, :1]),
                 dict(caches=[] if name != "copy" else [kw["caches"][0], kw["caches"][1][:5]])],
    }[name]
    from paged_kv_cache_76_gb300 import PAError
    for e in edits:
        with pytest.raises((ValueError, TypeError, AttributeError, PAError)):
            f(**{**kw, **e})
    assert ops.get_device_error() == 0


@pytest.mark.gpu
def test_a_given_output_and_refusals_of_the_c_call(taken):
    from paged_kv_cache_76_gb300 import PAError
    f, kw = calls("cuda")["decode"]
    out = torch.zeros_like(kw["q"])
    assert f(**kw, out=out) is out and torch.equal(out, f(**kw))
    assert taken == [True, True]
    with pytest.raises(PAError):
        f(**kw, split_tokens=33)
    f, kw = calls("cuda")["prefill"]
    with pytest.raises(PAError):
        f(**{**kw, "scale": 0.0})
    f, kw = calls("cuda")["fork"]
    with pytest.raises(PAError):
        f(**{**kw, "block_size": 5})
    assert taken == [True] * 5


@pytest.mark.gpu
@pytest.mark.parametrize("name", ["fork", "dequantize"])
@pytest.mark.parametrize("inference", [False, True])
def test_outputs_of_one_allocation_are_tensors_of_their_own(name, inference, taken):
    f, kw = calls("cuda")[name]
    with torch.inference_mode(inference):
        out = f(**kw)
        assert taken == [True]
        want = [t.clone() for t in out]
        ends = sorted((t.data_ptr(), t.data_ptr() + t.numel() * t.element_size()) for t in out if t.numel())
        assert all(a[1] <= b[0] for a, b in zip(ends, ends[1:]))
        for i, t in enumerate(out):
            assert t.is_contiguous() and t.data_ptr() % 16 == 0 and not t.requires_grad and t.is_inference() == inference
            t.zero_()
            assert all(torch.equal(a, b) for a, b in zip(out[i + 1:], want[i + 1:]))
