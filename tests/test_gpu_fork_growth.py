"""fork_blocks asked for more pages than 32 bits count: as for more than there are, the new batch is empty."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def ops():
    from paged_kv_cache_76_gb300 import _lib, ops
    try:
        _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
    torch.cuda.init()
    yield ops
    torch.cuda.empty_cache()


def test_more_pages_than_32_bits_count(ops):
    rows, bs, width = 9, 4, 2 ** 28 - 1  # nine rows of 2^28 - 1 pages: 2^31 and more
    grow = width * bs
    torch.cuda.empty_cache()
    if torch.cuda.mem_get_info()[0] < rows * (4 * (width + grow) + grow) + (8 << 30):
        pytest.skip("tables and slots of a thousand million tokens a row")

    def i32(*shape):
        return torch.zeros(*shape, dtype=torch.int32, device="cuda")
    held = i32(1, 2)
    held[0, 1] = 5
    tables, lens, pairs, slots, left = ops.fork_blocks(held, i32(1) + 7, i32(rows) - 1, 1000, bs, grow=grow,
                                                       max_blocks=width)
    assert ops.get_device_error() == 10
    assert left.tolist() == [1000] and torch.count_nonzero(lens) == 0 and bool((pairs == -1).all())
    for r in range(rows):
        assert bool((tables[r] == -1).all()) and bool((slots[r] == -1).all())
    # the same rows, one of them with a sequence: what it takes is as ever
    del tables, slots
    few = ops.fork_blocks(held, i32(1) + 7, i32(rows) - 2, 1000, bs, grow=3)
    assert few[4].tolist() == [1000] and ops.get_device_error() == 0
