"""The calls of the 4-bit cache and of forked pages together, as a program that
samples several continuations of its prompts makes them, without the host
knowing a page: prompts taken in by chunks (fork_blocks, quantize_and_cache,
chunked_prefill_kv4), steps at which beams go on from others, end and begin
(fork_blocks, copy_pages, decode_kv4), and drafted tokens verified.  A second
layer keeps its keys and values in 16 bits under the same tables
(reshape_and_cache, decode), and an encoder's pages are pinned in the same pool.

A float64 model follows along: per sequence the rows it has written, quantised
as the definition says for the first layer.  Tolerances as in test_gpu_kv4.py;
for the second layer as in test_gpu_moved_cache_run.py."""
import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu
HQ, HKV, D = 8, 2, 128
G = HQ // HKV
SCALE = D ** -0.5
NB = 96


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_76_gb300 import _lib
    try:
        _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
    torch.cuda.init()


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


class Program:
    def __init__(self, seed, bs, dtype):
        from paged_kv_cache_76_gb300 import ops
        self.ops, self.bs, self.dtype = ops, bs, dtype
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        # whatever a page held before, NaN
        self.small = [torch.full_like(ops.kv4_cache(NB, bs, HKV, D), 0xFF) for _ in range(2)]
        self.big = [torch.full((NB, bs, HKV, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2)]
        self.pinned = torch.zeros(NB, dtype=torch.bool, device="cuda")
        self.held = self.rng.choice(NB, 5, replace=False)
        self.pinned[torch.from_numpy(self.held).cuda()] = True
        self.frozen = [c[self.pinned].clone() for c in self.small + self.big]
        self.width = 24
        self.tables, self.lens = i32(np.full((1, self.width), -1)), i32([0])
        self.rows = [None]  # per row: four float64 [n, HKV, D], K and V of either layer; None: no sequence

    def go_on(self, parents, grow):
        """The next batch: pages, and new tokens' K and V written.  Returns the tokens' queries, packed by rows."""
        ops, most = self.ops, max(grow)
        out = ops.fork_blocks(self.tables, self.lens, i32(parents), NB, self.bs, grow=i32(grow), max_grow=most,
                              pinned=self.pinned)
        self.tables, self.lens, pairs, slots, self.free = out
        ops.copy_pages(self.small, pairs)
        ops.copy_pages(self.big, pairs)
        new = [None if p < -1 else [torch.zeros(0, HKV, D, dtype=torch.float64, device="cuda")] * 4 if p < 0
               else self.rows[p] for p in parents]
        grow = [0 if r is None else n for r, n in zip(new, grow)]
        T = sum(grow)
        kv = torch.randn(T, 2 * HKV * D, generator=self.gen, device="cuda").to(self.dtype)
        k, v = (x.unflatten(1, (HKV, D)) for x in kv.chunk(2, 1))
        # one slot mapping for the batch, padding and all
        flat = slots.flatten()
        at = torch.zeros(flat.numel(), dtype=torch.int64, device="cuda")
        where = [r * most + i for r, n in enumerate(grow) for i in range(n)]
        at[torch.tensor(where, device="cuda")] = torch.arange(T, device="cuda")
        ops.quantize_and_cache(k[at], v[at], flat, *self.small)
        ops.reshape_and_cache(k[at], v[at], flat, *self.big)
        four = [ref.quantized(k)[0].cuda(), ref.quantized(v)[0].cuda(), k.double(), v.double()]
        done = 0
        for i, r in enumerate(new):
            if r is not None:
                new[i] = [torch.cat([a, b[done:done + grow[i]]]) for a, b in zip(r, four)]
                done += grow[i]
        self.rows = new
        want = [0 if r is None else len(r[0]) for r in new]
        assert self.lens.tolist() == want
        used = {b for t, n in zip(self.tables.tolist(), want) for b in t[:-(-n // self.bs)]}
        assert not used & set(self.held.tolist())
        assert self.free.item() == NB - len(used) - len(self.held)
        return torch.randn(T, HQ, D, generator=self.gen, device="cuda").mul_(2).to(self.dtype), grow

    def check(self, got, q, row, seen, layer):
        """One query's outputs [HQ, D] against the model's first `seen` tokens of a row."""
        u = torch.finfo(self.dtype).eps / 2
        weight = 2.0 ** -11 if layer == 0 else u
        for h in range(HKV):
            k, v = (self.rows[row][2 * layer + i][:, h] for i in range(2))
            x = q[h * G:(h + 1) * G].double()
            mask = (torch.arange(len(k), device="cuda") < seen)[None].expand(G, -1)
            want, size = ref.attend(x, k, v, SCALE, mask)
            err = (D + 4) * 2.0 ** -24 * SCALE * (x.abs() @ k.abs().T).amax(-1, keepdim=True)
            tol = 2 * u * want.abs() + (weight + 2.0 ** -19 + 4 * err) * size + 1e-6
            assert bool(((got[h * G:(h + 1) * G].double() - want).abs() <= tol).all()), (row, h, layer)

    def prompts(self, parents, grow):
        q, grow = self.go_on(parents, grow)
        start = np.concatenate([[0], np.cumsum(grow)])
        out = self.ops.chunked_prefill_kv4(q, i32(start), self.lens, *self.small, self.tables, SCALE, max(grow))
        for r, n in enumerate(grow):
            for i in range(n):
                self.check(out[start[r] + i], q[start[r] + i], r, len(self.rows[r][0]) - n + i + 1, 0)

    def step(self, parents):
        q, grow = self.go_on(parents, [1] * len(parents))
        rows = torch.zeros(len(parents), HQ, D, dtype=self.dtype, device="cuda")
        live = [r for r, n in enumerate(grow) if n]
        rows[torch.tensor(live, device="cuda")] = q
        four = self.ops.decode_kv4(rows, *self.small, self.tables, self.lens, SCALE)
        whole = self.ops.decode(rows, *self.big, self.tables, self.lens, SCALE)
        for r, n in enumerate(grow):
            if n:
                self.check(four[r], rows[r], r, len(self.rows[r][0]), 0)
                self.check(whole[r], rows[r], r, len(self.rows[r][0]), 1)
            else:
                assert torch.count_nonzero(four[r]) == 0

    def drafts(self, parents, n):
        q, grow = self.go_on(parents, [n] * len(parents))
        assert grow == [n] * len(parents)
        out = self.ops.decode_kv4(q.view(len(parents), n, HQ, D), *self.small, self.tables, self.lens, SCALE)
        for r in range(len(parents)):
            for i in range(n):
                self.check(out[r, i], q[r * n + i], r, len(self.rows[r][0]) - (n - 1 - i), 0)


@pytest.mark.parametrize("seed,bs,dtype", [(0, 16, torch.bfloat16), (1, 8, torch.float16), (2, 32, torch.bfloat16)])
def test_a_program_that_samples(seed, bs, dtype):
    p = Program(seed, bs, dtype)
    p.prompts([-1, -1, -1], [37, 64, 5])
    p.prompts([0, 1, 2], [20, 33, 11])                 # the prompts' second chunks
    p.step([0, 0, 0, 1, 1, 2])                         # samples of each prompt: they share its pages
    for _ in range(3):
        p.step([int(p.rng.integers(0, 3)) for _ in range(3)] + [int(p.rng.integers(3, 5)) for _ in range(2)] + [5])
    p.drafts([0, 1, 1, 3, 4, 5], 4)
    p.step([0, 1, -2, 3, 3, 5, -1])                    # one ends, one begins, one is continued twice
    p.drafts([0, 1, 3, 4, 5, 6], 3)
    free = p.free.item()
    p.step([0, -2, -2, -2, 4, 5])
    assert p.free.item() >= free                       # what they held has come back
    for c, f in zip(p.small + p.big, p.frozen):        # pinned pages as they were, bit for bit
        assert torch.equal(c[p.pinned].view(torch.uint8), f.view(torch.uint8))
    assert p.ops.get_device_error() == 0
