"""fork_blocks against the host's row-by-row form (whole numbers: equal), and
copy_pages against indexing."""
import numpy as np
import pytest
import torch

import fork_ref

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
    return ops


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def check(ops, tables, lens, parents, grow, num_blocks, bs, width, max_grow=None, pinned=(), error=0):
    """Both forms; `grow` a count or a list.  Returns the device's outputs."""
    mask = torch.zeros(num_blocks, dtype=torch.bool, device="cuda")
    mask[list(pinned)] = True
    t, n, p = i32(tables), i32(lens), i32(parents)
    keep = t.clone(), n.clone()
    if isinstance(grow, int):
        got = ops.fork_blocks(t, n, p, num_blocks, bs, grow=grow, pinned=mask if pinned else None, max_blocks=width)
        grow, max_grow = [grow] * len(parents), grow
    else:
        got = ops.fork_blocks(t, n, p, num_blocks, bs, grow=i32(grow), max_grow=max_grow,
                              pinned=mask.to(torch.uint8) if pinned else None, max_blocks=width)
    assert ops.get_device_error() == error
    want = fork_ref.fork(tables.tolist() if hasattr(tables, "tolist") else tables, list(lens), list(parents), list(grow),
                         num_blocks, bs, width, max_grow, pinned)
    names = ("tables", "lens", "pairs", "slots")
    for name, g, w in zip(names, got, want):
        w = torch.tensor(np.asarray(w).reshape(tuple(g.shape)), dtype=torch.int32)
        assert torch.equal(g.cpu(), w), name
    assert got[4].tolist() == [want[4]]
    assert torch.equal(t, keep[0]) and torch.equal(n, keep[1])
    return got


def batch(rng, rows, bs, hi, num_blocks, share):
    """Tables of rows of which some share leading blocks; lengths 0 to hi."""
    width = -(-hi // bs)
    lens = rng.integers(0, hi + 1, rows)
    lens[rng.random(rows) < 0.2] = rng.integers(0, width + 1) * bs
    lens = np.minimum(lens, hi)
    perm = list(rng.permutation(num_blocks))
    tables = np.full((rows, width), -5)
    for r in range(rows):
        n = -(-int(lens[r]) // bs)
        k = 0
        if r and rng.random() < share:
            other = int(rng.integers(0, r))
            k = int(min(n, -(-int(lens[other]) // bs), rng.integers(0, width + 1)))
            tables[r, :k] = tables[other, :k]
        tables[r, k:n] = [perm.pop() for _ in range(n - k)]
    return tables, lens


@pytest.mark.parametrize("seed", range(12))
def test_any_batch(ops, seed):
    rng = np.random.default_rng(seed)
    bs = int(rng.choice([4, 8, 16, 32]))
    rows, new = int(rng.integers(1, 40)), int(rng.integers(1, 60))
    hi = int(rng.integers(1, 300))
    num_blocks = rows * (hi // bs + 2) + 4 * new + 10
    tables, lens = batch(rng, rows, bs, hi, num_blocks, 0.6)
    parents = rng.integers(-3, rows, new)
    pinned = rng.choice(num_blocks, 3, replace=False).tolist() if seed % 2 else ()
    width = tables.shape[1] + 2
    if seed % 3:
        check(ops, tables, lens, parents, rng.integers(0, 9, new).tolist(), num_blocks, bs, width, 8, pinned)
    else:
        check(ops, tables, lens, parents, int(rng.integers(0, 3)), num_blocks, bs, width, None, pinned)


def test_beams_share_copy_and_give_back(ops):
    # a prompt of 6 tokens (blocks 4, 9), three rows after it; bs 4
    t = [[4, 9, -1], [4, 9, -1], [7, 3, -1]]
    # rows 0 and 1 both go on inside block 9; row 2 is dropped, its blocks come back
    got = check(ops, np.array(t), [6, 6, 7], [0, 1, 0], 1, 10, 4, 3)
    assert got[0].tolist() == [[4, 9, -1], [4, 0, -1], [4, 1, -1]]
    assert got[2].tolist() == [[-1, -1], [9, 0], [9, 1]]
    assert got[3].tolist() == [[9 * 4 + 2], [2], [6]]
    # a row that does not grow holds the page: the writer copies
    got = check(ops, np.array(t), [6, 6, 7], [0, 1], [0, 2], 10, 4, 3, 2)
    assert got[2].tolist() == [[-1, -1], [9, 0]]
    # a full last block: shared, a fresh one behind it
    got = check(ops, np.array(t), [8, 8, 7], [0, 0], 1, 10, 4, 3)
    assert got[0].tolist() == [[4, 9, 0], [4, 9, 1]]
    # pinned: the only writer copies too
    check(ops, np.array(t), [6, 6, 7], [2], 1, 10, 4, 3, None, (3,))
    # a shorter row that would go on inside a block that a longer one has filled
    check(ops, np.array([[4, 9], [4, 9]]), [6, 8], [0, 1], 1, 10, 4, 3)


def test_new_sequences_and_none(ops):
    none = np.full((1, 2), -1)
    got = check(ops, none, [0], [-1, -2, -1, 0], [9, 5, 0, 3], 8, 4, 4, 9)
    assert got[1].tolist() == [9, 0, 0, 3] and got[4].tolist() == [4]
    check(ops, none, [0], [-2, -7], 1, 8, 4, 2)
    # no rows before, none after
    got = ops.fork_blocks(i32(np.zeros((0, 2))), i32([]), i32([-1, -1]), 8, 4, grow=5)
    assert got[0].tolist() == [[0, 1], [2, 3]] and got[4].tolist() == [4]
    got = ops.fork_blocks(i32([[3, 1]]), i32([8]), i32([]), 8, 4, grow=1)
    assert got[4].tolist() == [8] and got[0].shape == (0, 2)
    assert ops.get_device_error() == 0


def test_too_few_blocks_leave_everything_as_it_was(ops):
    t = np.array([[0, 1], [2, 3]])
    check(ops, t, [7, 8], [0, 0, 1], 1, 5, 4, 3, error=10)      # a copy and a fresh one: 1 free
    got = check(ops, t, [7, 8], [0, 0], 1, 5, 4, 3)             # row 1's blocks come back
    assert got[4].tolist() == [2]
    check(ops, t, [7, 8], [0, 1], 0, 4, 4, 2)                   # nothing needed, nothing free
    check(ops, t, [7, 8], [-1] * 3, 12, 4, 4, 4, error=10)


def test_rows_in_error_are_rows_without_a_sequence(ops):
    t = np.array([[0, 1], [2, 3]])
    check(ops, t, [7, 8], [0, 2, 1], 1, 8, 4, 3, error=9)           # no such parent
    check(ops, t, [7, 9], [0, 1], 1, 8, 4, 3, error=2)              # a length past its table
    check(ops, t, [7, -1], [0, 1], 1, 8, 4, 3, error=2)
    check(ops, t, [7, 8], [0, 1], 1, 8, 4, 2, error=2)              # a new length past the new table
    check(ops, t, [7, 8], [0, 1, 0], [1, -1, 9], 8, 4, 3, 8, error=9)
    check(ops, np.array([[0, 99], [-4, 3]]), [7, 8], [0, 1, 0], 1, 8, 4, 3, error=1)


@pytest.mark.parametrize("rows,new,width,num_blocks", [(600, 700, 513, 5000), (8, 16, 8191, 300000), (1, 3, 70000, 70100)])
def test_large_batches(ops, rows, new, width, num_blocks):
    """More than a cluster takes: a launch per step."""
    rng = np.random.default_rng(rows)
    bs = 4
    lens = rng.integers(0, min(width, num_blocks // max(rows, 2) * 2) * bs, rows)
    tables = np.full((rows, width), -1)
    for r in range(rows):
        n = -(-int(lens[r]) // bs)
        tables[r, :n] = rng.integers(0, num_blocks * 2 // 3, n)  # shared in any way
    parents = rng.integers(-2, rows, new)
    check(ops, tables, lens, parents, rng.integers(0, 4, new).tolist(), num_blocks, bs, width + 1, 3)


@pytest.mark.parametrize("num_blocks", [6000, 90000])
def test_growth_by_whole_prompts(ops, num_blocks):
    """Rows that take up to 1300 pages at a time, round scattered pinned ones, down to the last page of the pool."""
    rng = np.random.default_rng(num_blocks)
    bs, parents, grow = 4, [-1, 0, 0, -1, 1, -2, -1], [5200, 2049, 1, 130, 0, 0, 7]
    lens = [2046, 9]
    held = rng.permutation(num_blocks)[:515]
    tables = np.full((2, 512), -1)
    tables[0], tables[1, :3] = held[:512], held[512:]
    free = np.setdiff1d(np.arange(num_blocks), held)
    pinned = rng.permutation(free)[:len(free) // 3].tolist()
    pinned += [int(held[0]), int(held[514])]
    got = check(ops, tables, lens, parents, grow, num_blocks, bs, 1500, 5200, pinned)
    left = int(got[4])
    assert left > 0
    # the same with all but the pages that it takes pinned: none left; with one more: too few
    used = set(got[0].flatten().tolist()) - {-1}
    rest = [int(b) for b in np.setdiff1d(free, list(used))]
    check(ops, tables, lens, parents, grow, num_blocks, bs, 1500, 5200, sorted(set(pinned) | set(rest)))
    last = max(used - set(held.tolist()))
    check(ops, tables, lens, parents, grow, num_blocks, bs, 1500, 5200, sorted(set(pinned) | set(rest) | {last}), error=10)


def test_many_rows(ops):
    rng = np.random.default_rng(5)
    rows, bs, num_blocks = 65535, 4, 70000
    lens = rng.integers(0, 5, rows)
    tables = np.full((rows, 1), -1)
    tables[:, 0] = np.arange(rows)
    parents = rng.permutation(rows)
    check(ops, tables, lens, parents, 0, num_blocks, bs, 1)


def test_copies_in_every_cache(ops):
    gen = torch.Generator(device="cuda").manual_seed(1)
    pairs = i32([[3, 0], [-1, -1], [5, 7], [3, 2], [-1, 9]])
    for shape, dtype, n in [((10, 16, 8, 128), torch.bfloat16, 4), ((10, 4, 4 * 36), torch.uint8, 70),
                            ((10, 4, 1, 64), torch.float16, 1), ((10, 32, 3, 128), torch.bfloat16, 65)]:
        caches = [torch.randint(0, 200, shape, generator=gen, device="cuda").to(dtype) for _ in range(n)]
        want = [c.clone() for c in caches]
        for c in want:
            c[[0, 7, 2]] = c[[3, 5, 3]]
        ops.copy_pages(caches, pairs)
        assert all(torch.equal(a, b) for a, b in zip(caches, want))
        assert ops.get_device_error() == 0
    ops.copy_pages(caches, i32([[1, 10], [10, 1], [2, -1], [4, 8]]))
    assert ops.get_device_error() == 1
    for c in want:
        c[8] = c[4]
    assert all(torch.equal(a, b) for a, b in zip(caches, want))
    ops.copy_pages([], pairs)
    ops.copy_pages(caches, pairs[:0])


def test_captured_and_on_another_stream(ops):
    rng = np.random.default_rng(2)
    tables, lens = batch(rng, 9, 4, 60, 400, 0.5)
    t, n = i32(tables), i32(lens)
    parents = i32(rng.integers(-1, 9, 12))
    cache = torch.randn(400, 4, 2, 64, device="cuda").to(torch.bfloat16)
    start = cache.clone()
    g = torch.cuda.CUDAGraph()
    side = torch.cuda.Stream()
    with torch.cuda.graph(g):
        out = ops.fork_blocks(t, n, parents, 400, 4)
        ops.copy_pages([cache], out[2])
    for seed in range(3):
        parents.copy_(i32(rng.integers(-1, 9, 12)))
        cache.copy_(start)
        g.replay()
        after = cache.clone()
        cache.copy_(start)
        side.wait_stream(torch.cuda.current_stream())
        want = ops.fork_blocks(t, n, parents, 400, 4, stream=side)
        ops.copy_pages([cache], want[2], stream=side)
        torch.cuda.current_stream().wait_stream(side)
        assert all(torch.equal(a, b) for a, b in zip(out, want))
        assert torch.equal(after, cache)
    assert ops.get_device_error() == 0


def test_a_large_batch_captured_and_two_at_once(ops):
    """The cooperative form in a graph, and two calls on two streams."""
    rng = np.random.default_rng(9)
    batches = []
    for seed in range(2):
        tables, lens = batch(rng, 300, 4, 900, 90000, 0.7)
        batches.append((i32(tables), i32(lens), i32(rng.integers(-1, 300, 400))))
    want = [ops.fork_blocks(*b, 90000, 4, grow=2, max_blocks=226) for b in batches]
    graphs, outs = [], []
    for b in batches:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(ops.fork_blocks(*b, 90000, 4, grow=2, max_blocks=226))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in range(2)]
    for _ in range(5):
        for o in outs:
            for x in o:
                x.fill_(-9)
        torch.cuda.synchronize()
        for s, g in zip(streams, graphs):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        for o, w in zip(outs, want):
            assert all(torch.equal(x, y) for x, y in zip(o, w))
    ws = torch.empty(8 << 20, dtype=torch.uint8, device="cuda")
    again = ops.fork_blocks(*batches[0], 90000, 4, grow=2, max_blocks=226, workspace=ws)
    assert all(torch.equal(x, y) for x, y in zip(again, want[0]))
    assert ops.get_device_error() == 0
