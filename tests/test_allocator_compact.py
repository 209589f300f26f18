"""pa_alloc_compact: a sequence shrinks in place (after an eviction, or to the
accepted path of a draft).  Random scripts on the C++ allocator and the oracle
must agree field by field, refused calls change nothing, and what left the
prefix cache is not found again."""
import numpy as np
import pytest

from oracle.block_pool import AllocError, NoFreeBlocks, SequenceManager
from paged_kv_cache_76_gb300 import _lib
from paged_kv_cache_76_gb300.allocator import BlockAllocator
from paged_kv_cache_76_gb300.allocator import NoFreeBlocks as CNoFree


@pytest.fixture(scope="module", autouse=True)
def built():
    try:
        _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()


def both(c, o, op, *args):
    got = []
    for t in (c, o):
        try:
            v = getattr(t, op)(*args)
            got.append(("ok", v.tolist() if isinstance(v, np.ndarray) else v))
        except (NoFreeBlocks, CNoFree):
            got.append(("nofree", None))
        except (AllocError, _lib.PAError):
            got.append(("err", None))
    assert got[0][0] == got[1][0], (op, args, got)
    if got[0][0] == "ok" and got[0][1] is not None:
        assert got[0][1] == got[1][1], (op, args)
    return got[0][0]


def assert_same(c, o):
    assert c.free_list() == o.free_list()
    assert [c.ref(b) for b in range(c.num_blocks)] == o.pool.ref_cnt
    assert [c.block_hash(b) for b in range(c.num_blocks)] == [
        h if o.pool.cached_block_hash_to_block.get(h) == b else None for b, h in enumerate(o.pool.block_hash)]
    for s in o.tables:
        assert c.block_table(s) == o.block_table(s) and c.seq_len(s) == o.num_tokens[s]
    assert c.stats()["waste_slots"] == sum(o.waste(s) for s in o.tables)


@pytest.mark.parametrize("seed", range(8))
def test_random_scripts_match_the_oracle(seed):
    rng = np.random.default_rng(seed)
    nb, bs = int(rng.integers(10, 60)), int(rng.choice([1, 2, 4, 16]))
    c, o = BlockAllocator(nb, bs), SequenceManager(nb, bs)
    if seed % 4:
        c.enable_prefix_caching(), o.enable_prefix_caching()
    if seed % 2:
        c.enable_swap(nb), o.enable_swap(nb)
    live, nxt, done = [], 0, 0
    for _ in range(700):
        kind = rng.choice(["add", "append", "tokens", "tokens", "share", "cow", "free", "compact", "compact", "cut",
                           "swap_out", "swap_in"])
        if kind == "add" or not live:
            prompt = rng.integers(0, 3, size=int(rng.integers(0, 4 * bs))).tolist()
            both(c, o, "add_seq_cached", nxt, prompt, 0)
            live.append(nxt)
            nxt += 1
        else:
            s = int(rng.choice(live))
            L = o.num_tokens[s]
            if kind == "append":
                both(c, o, "append_slots", s, int(rng.integers(0, 2 * bs + 2)))
            elif kind == "tokens":
                both(c, o, "append_tokens", s, rng.integers(0, 3, size=int(rng.integers(0, 2 * bs + 2))).tolist())
            elif kind == "share":
                both(c, o, "add_seq", nxt)
                both(c, o, "share", nxt, s, int(rng.integers(0, L + 1)))
                live.append(nxt)
                nxt += 1
            elif kind == "cow":
                both(c, o, "cow", s, int(rng.integers(-1, len(o.tables[s]) + 1)))
            elif kind == "free":
                both(c, o, "free_seq", s)
                live.remove(s)
            elif kind == "compact":
                n = int(rng.integers(0, L + 2))
                done += both(c, o, "compact", s, int(rng.integers(-1, n + 1)), n) == "ok"
            elif kind == "cut":
                n = int(rng.integers(0, L + 1))
                done += both(c, o, "compact", s, n, n) == "ok"
            else:
                got = []
                for target in (c, o):
                    try:
                        getattr(target, kind)(s)
                        got.append("ok")
                    except (NoFreeBlocks, AllocError, _lib.PAError):
                        got.append("refused")
                assert got[0] == got[1], (kind, got)
        if not (seed % 2 and o.on_cpu):
            assert_same(c, o)
        if rng.random() < 0.02:
            w = c.export()
            assert BlockAllocator.from_words(w).export().tolist() == w.tolist()
    assert done > 20


def test_shared_blocks_are_refused_and_nothing_changes():
    c = BlockAllocator(16, 4)
    c.add_seq(0)
    c.append_slots(0, 10)
    c.add_seq(1)
    c.share(1, 0, 8)
    before = c.export().tolist()
    for first, n in ((0, 10), (3, 5), (7, 8)):
        with pytest.raises(_lib.PAError) as e:
            c.compact(0, first, n)
        assert e.value.status == _lib.PA_ERR_SHARED_BLOCK
    for first, n in ((-1, 4), (5, 4), (0, 11)):
        with pytest.raises(_lib.PAError) as e:
            c.compact(0, first, n)
        assert e.value.status == _lib.PA_ERR_INVALID
    with pytest.raises(_lib.PAError):
        c.compact(7, 0, 0)
    assert c.export().tolist() == before
    c.compact(0, 8, 9)                       # the private tail may be rewritten
    c.compact(0, 4, 4)                       # a truncation into the shared blocks releases the rest
    assert c.block_table(0) == [0] and c.ref(1) == 1 and c.seq_len(1) == 8


def test_rewritten_blocks_leave_the_prefix_cache():
    c = BlockAllocator(16, 4)
    c.enable_prefix_caching()
    prompt = list(range(12))
    assert c.add_seq_cached(0, prompt) == 0
    c.append_tokens(0, prompt)
    assert all(c.block_hash(b) is not None for b in c.block_table(0))
    first = c.block_table(0)[0]
    c.compact(0, 4, 9)                       # tokens 4..8 are others now; block 2 is cut
    assert c.block_hash(first) is not None and [c.block_hash(b) for b in c.block_table(0)[1:]] == [None, None]
    assert c.add_seq_cached(1, prompt) == 4  # only the untouched block is found
    c.append_tokens(0, [1, 2, 3, 4, 5])
    assert [c.block_hash(b) for b in c.block_table(0)[1:]] == [None] * 3   # unknown tokens: nothing registered
