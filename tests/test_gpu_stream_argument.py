"""Calls given a stream other than the current one: the scratch they allocate
belongs to that stream, so that nothing on the current one is handed the same
memory while the call has yet to run; and the results are the same."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF, HQ, HKV, D, BS = torch.bfloat16, 8, 2, 128, 16


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_76_gb300 import _lib
    try:
        _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
    torch.cuda.init()


def calls():
    """name -> (function, arguments, position of the scratch's pointer among the C call's arguments or None)"""
    from paged_kv_cache_76_gb300 import ops
    g = torch.Generator(device="cuda").manual_seed(8)

    def x(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(BF)

    def i32(a):
        return torch.tensor(a, dtype=torch.int32, device="cuda")

    kc, vc = x(128, BS, HKV, D), x(128, BS, HKV, D)
    tables = torch.arange(128, dtype=torch.int32, device="cuda").view(2, 64)
    lens, q, kv = i32([1000, 700]), x(2, HQ, D), dict(k_cache=kc, v_cache=vc)
    at = dict(**kv, block_tables=tables, context_lens=lens, scale=0.09)
    shared = tables.clone()
    shared[1, :8] = tables[0, :8]            # both requests begin with the prefix
    scores = torch.rand(2, HKV, 1024, generator=g, device="cuda")
    return {
        "decode": (ops.decode, dict(q=q, **at, split_tokens=64), 14),
        "verify": (ops.verify_decode, dict(q=x(2, 3, HQ, D), **at, split_tokens=64), 15),
        "verify_tc": (ops.verify_decode_tc, dict(q=x(2, 3, HQ, D), **at), None),
        "prefix": (ops.decode_shared_prefix, dict(**{**at, "block_tables": shared}, q=q, prefix_len=128,
                                                  prefix_blocks=tables[0, :8].contiguous()), 16),
        "prefill": (ops.chunked_prefill, dict(q=x(7, HQ, D), q_start=i32([0, 4, 7]), max_q_len=4, **at), None),
        "rope": (ops.norm_rope_and_cache, dict(
            q=q, k=x(2, HKV, D), v=x(2, HKV, D), positions=i32([5, 6]), cos_sin=ops.rope_table(32, 64, device="cuda"),
            slot_mapping=i32([2040, 2041]), **kv), None),
        "tree": (ops.verify_tree, dict(
            q=x(7, HQ, D), q_start=i32([0, 4, 7]), max_q_len=4, split_tokens=128, **at,
            tree_mask=torch.cat([ops.tree_mask([-1, 0, 0, 1]), ops.tree_mask([-1, 0, 1])]).cuda()), 18),
        "accumulate": (ops.decode_accumulate, dict(q=q, **at, scores=scores), 19),
        "select": (ops.evict_select, dict(scores=scores, context_lens=lens, sink=2, heavy=200, recent=50), None),
    }


NAMES = ["decode", "verify", "verify_tc", "prefix", "prefill", "rope", "tree", "accumulate", "select"]


@pytest.mark.parametrize("name", [n for n in NAMES if n not in ("verify_tc", "prefill", "rope", "select")])
def test_scratch_is_the_streams_own(name, monkeypatch):
    """Nothing is launched here: only who is handed the memory is looked at."""
    from paged_kv_cache_76_gb300 import ops
    f, kw, at = calls()[name]
    seen = []
    monkeypatch.setattr(ops, "_launch", lambda fn, *args: seen.append(args))
    for stream in (torch.cuda.Stream(), torch.cuda.ExternalStream(torch.cuda.Stream().cuda_stream)):
        seen.clear()
        held = f(**kw, stream=stream)               # else the results are free again, too
        scratch, size = seen[0][at], seen[0][at + 1]
        assert scratch and size > 0
        mine = [torch.empty(size, dtype=torch.uint8, device="cuda") for _ in range(4)]
        assert all(not t.data_ptr() <= scratch < t.data_ptr() + size for t in mine)
        with torch.cuda.stream(stream):
            again = torch.empty(size, dtype=torch.uint8, device="cuda")
        assert again.data_ptr() == scratch          # freed, for the stream's own next use
        del held, mine, again


@pytest.mark.parametrize("name", NAMES)
def test_results_are_those_of_the_current_stream(name):
    from paged_kv_cache_76_gb300 import ops
    f, kw, _ = calls()[name]
    inputs = {k: t.clone() for k, t in kw.items() if isinstance(t, torch.Tensor)}
    side = torch.cuda.Stream()

    def run(**more):
        args = {**kw, **{k: t.clone() for k, t in inputs.items()}}
        torch.cuda.synchronize()
        if more:
            with torch.cuda.stream(side):
                torch.cuda._sleep(2_000_000)        # a millisecond: the host is far ahead
        r = f(**args, **more)
        for _ in range(4):                          # what the current stream is handed meanwhile
            torch.full((1 << 20,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.current_stream().wait_stream(side)
        out = list(r) if isinstance(r, tuple) else [r]
        got = [t.clone() for t in out + [t for t in args.values() if isinstance(t, torch.Tensor)]]
        torch.cuda.synchronize()
        return got

    want, got = run(), run(stream=side)
    assert ops.get_device_error() == 0
    assert all(torch.equal(a, b) for a, b in zip(want, got))
