"""A cached block that a sequence holds in part leaves the prefix cache when the
sequence, its last owner, writes behind its tokens: the block's hash names
tokens that it then no longer holds."""
import pytest

from oracle.block_pool import SequenceManager
from paged_kv_cache_76_gb300 import _lib
from paged_kv_cache_76_gb300.allocator import BlockAllocator


@pytest.fixture(scope="module", autouse=True)
def built():
    try:
        _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()


@pytest.mark.parametrize("make", [BlockAllocator, SequenceManager])
@pytest.mark.parametrize("how", ["cut while shared", "shared in part"])
@pytest.mark.parametrize("write", ["append_slots", "append_tokens", "cow first"])
def test_a_partly_held_block_is_not_found_after_a_write(make, how, write):
    a, prompt = make(16, 4), list(range(8))
    a.enable_prefix_caching()
    a.add_seq_cached(0, prompt, 0)
    a.append_tokens(0, prompt)              # two full blocks, both cached
    a.add_seq(1)
    if how == "cut while shared":
        a.share(1, 0, 8)
        a.compact(0, 6, 6)                  # 1 still reads the whole block
        keeps = 0
    else:
        a.share(1, 0, 6)
        keeps = 1
    assert a.add_seq_cached(2, prompt + [8], 0) == 8
    a.free_seq(2)
    a.free_seq(1 - keeps)                   # the other owner goes: the block is private, and still right
    assert a.add_seq_cached(3, prompt + [8], 0) == 8
    with pytest.raises(Exception):          # shared again, with 3: not to be written
        a.append_slots(keeps, 1)
    assert a.add_seq_cached(4, prompt + [8], 0) == 8
    a.free_seq(3), a.free_seq(4)
    b = a.block_table(keeps)[1]
    if write == "cow first":
        assert tuple(a.cow(keeps, 1)) == (b, b)
        write = "append_slots"
    slots = a.append_slots(keeps, 1) if write == "append_slots" else a.append_tokens(keeps, [77])
    assert list(slots) == [4 * b + 2]
    assert a.add_seq_cached(5, prompt + [8], 0) == 4    # the first block alone


def test_an_append_that_is_refused_keeps_the_block_cached():
    a, prompt = BlockAllocator(2, 4), list(range(8))
    a.enable_prefix_caching()
    a.add_seq_cached(0, prompt, 0)
    a.append_tokens(0, prompt)
    a.add_seq(1)
    a.share(1, 0, 6)
    a.free_seq(0)
    before = a.export().tolist()
    with pytest.raises(Exception):
        a.append_slots(1, 3)                # a block more than there is
    after = a.export().tolist()
    assert [x for x, y in zip(before, after) if x != y] in ([], [0])   # at most the count of failures
    assert a.block_hash(a.block_table(1)[1]) is not None
