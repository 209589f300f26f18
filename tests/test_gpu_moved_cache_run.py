"""The calls for caches whose slot order is not the position order, together as
a serving loop makes them: new tokens normed, rotated and written; decode steps
that keep score; an eviction to a budget (select, compact, release of blocks);
a drafted tree verified and its accepted path kept; and decoding on over what
is left.  A float64 model of every sequence and KV head follows along: it takes
each written row as the cache holds it, and from then on moves rows by itself.

Tolerances as in test_gpu_verify_tree.py (outputs) and test_gpu_eviction.py
(scores, summed over the steps)."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

BS, HQ, HKV, D = 16, 8, 2, 128
G = HQ // HKV
DT = torch.bfloat16
SCALE = 1 / np.sqrt(D)


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


class Loop:
    def __init__(self, seed, seqs, dtype=DT):
        from paged_kv_cache_76_gb300 import ops
        from paged_kv_cache_76_gb300.allocator import BlockAllocator
        self.ops, self.seqs, self.dtype = ops, seqs, dtype
        self.rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        self.alloc = BlockAllocator(60, BS, self.rng.permutation(60))
        self.kc, self.vc = (torch.full((60, BS, HKV, D), float("nan"), dtype=dtype, device="cuda") for _ in range(2))
        self.table = ops.rope_table(4096, D, device="cuda")
        self.qw, self.kw = ((1 + 0.1 * torch.randn(D, generator=self.gen, device="cuda")).to(dtype) for _ in range(2))
        self.scores = torch.zeros(len(seqs) + 2, HKV, 640, device="cuda")
        self.rows = i32(self.rng.permutation(len(seqs) + 2)[:len(seqs)])
        self.next_pos = [0] * len(seqs)
        # the model: per sequence and KV head the rows of K and V and the scores, float64
        self.k = [[torch.zeros(0, D, dtype=torch.float64, device="cuda") for _ in range(HKV)] for _ in seqs]
        self.v = [[torch.zeros(0, D, dtype=torch.float64, device="cuda") for _ in range(HKV)] for _ in seqs]
        self.s = [[torch.zeros(0, dtype=torch.float64, device="cuda") for _ in range(HKV)] for _ in seqs]
        self.s_tol = 0.0
        for s in seqs:
            self.alloc.add_seq(s)

    def write(self, positions):
        """positions[r]: those of sequence r's new tokens.  Returns their rotated queries, packed."""
        counts = [len(p) for p in positions]
        slots = np.concatenate([self.alloc.append_slots(s, n) for s, n in zip(self.seqs, counts)])
        T = sum(counts)
        qkv = torch.randn(T, (HQ + 2 * HKV) * D, generator=self.gen, device="cuda").to(self.dtype)
        q, k, v = (x.unflatten(1, (h, D)) for x, h in zip(qkv.split([HQ * D, HKV * D, HKV * D], 1), (HQ, HKV, HKV)))
        out = self.ops.norm_rope_and_cache(q, k, v, i32(np.concatenate(positions)), self.table, i32(slots), self.kc,
                                           self.vc, q_weight=self.qw, k_weight=self.kw)
        at = torch.from_numpy(slots).long().cuda()
        rows = [c.view(-1, HKV, D)[at].double() for c in (self.kc, self.vc)]
        done = 0
        for r, n in enumerate(counts):
            for h in range(HKV):
                self.k[r][h] = torch.cat([self.k[r][h], rows[0][done:done + n, h]])
                self.v[r][h] = torch.cat([self.v[r][h], rows[1][done:done + n, h]])
                self.s[r][h] = torch.cat([self.s[r][h], torch.zeros(n, dtype=torch.float64, device="cuda")])
            done += n
        return out

    def tables(self):
        width = max(max(len(self.alloc.block_table(s)) for s in self.seqs), 1)
        t, lens = self.alloc.build_tables(self.seqs, width)
        return torch.from_numpy(t).cuda(), torch.from_numpy(lens).cuda()

    def check(self, got, q, r, h, seen):
        """One output row against the model; returns the weights."""
        k, v = self.k[r][h // G][seen], self.v[r][h // G][seen]
        x = q.double()
        p = torch.softmax(k @ x * SCALE, 0)
        u = torch.finfo(self.dtype).eps / 2
        err = (D + 4) * 2.0 ** -24 * SCALE * float((k.abs() @ x.abs()).max())
        want = p @ v
        tol = 2 * u * want.abs() + (u + 2 * err + 2.0 ** -20) * (p @ v.abs()) + 1e-7
        assert bool(((got.double() - want).abs() <= tol).all()), (r, h)
        return p, 2 * err + 2.0 ** -16 + 2.0 ** -19

    def decode(self):
        q = self.write([[p] for p in self.next_pos])
        self.next_pos = [p + 1 for p in self.next_pos]
        tables, lens = self.tables()
        out, _ = self.ops.decode_accumulate(q, self.kc, self.vc, tables, lens, SCALE, self.scores,
                                            score_rows=self.rows)
        worst = 0.0
        for r in range(len(self.seqs)):
            for h in range(HQ):
                p, e = self.check(out[r, h], q[r, h], r, h, slice(None))
                self.s[r][h // G] += p
                worst = max(worst, e)
        self.s_tol += G * worst + 2.0 ** -20
        for r in range(len(self.seqs)):
            for g in range(HKV):
                n = len(self.s[r][g])
                mine = self.scores[int(self.rows[r]), g]
                assert torch.count_nonzero(mine[n:]) == 0
                assert float((mine[:n].double() - self.s[r][g]).abs().max()) <= self.s_tol

    def evict(self, sink, heavy, recent):
        tables, lens = self.tables()
        keep, n = self.ops.evict_select(self.scores, lens, sink, heavy, recent, score_rows=self.rows)
        budget = sink + heavy + recent
        for r in range(len(self.seqs)):
            L = int(lens[r])
            assert int(n[r]) == min(L, budget)
            for g in range(HKV):
                idx = keep[r, g, :int(n[r])].long()
                if L > budget:
                    mid = self.scores[int(self.rows[r]), g, sink:L - recent]
                    best = torch.sort(mid, descending=True, stable=True).indices[:heavy].sort().values + sink
                    want = torch.cat([torch.arange(sink, device="cuda"), best,
                                      torch.arange(L - recent, L, device="cuda")])
                    assert torch.equal(idx, want)
                self.k[r][g], self.v[r][g] = self.k[r][g][idx], self.v[r][g][idx]
                self.s[r][g] = self.s[r][g][idx]
        self.ops.compact_kv(self.kc, self.vc, tables, lens, keep, n, scores=self.scores, score_rows=self.rows)
        for r, s in enumerate(self.seqs):
            self.alloc.compact(s, min(sink, int(n[r])), int(n[r]))

    def tree(self, nodes):
        parents = [[int(self.rng.integers(max(-1, i - 3), i)) if i else -1 for i in range(n)] for n in nodes]
        depth = []
        for ps in parents:
            d = []
            for p in ps:
                d.append(d[p] + 1 if p >= 0 else 0)
            depth.append(d)
        base = [self.alloc.seq_len(s) for s in self.seqs]
        q = self.write([[self.next_pos[r] + x for x in d] for r, d in enumerate(depth)])
        tables, lens = self.tables()
        masks = [self.ops.tree_mask(p) for p in parents]
        start = np.concatenate([[0], np.cumsum(nodes)])
        out = self.ops.verify_tree(q, i32(start), torch.cat(masks).cuda(), lens, self.kc, self.vc, tables, SCALE,
                                   max(nodes))
        keep = np.full((len(self.seqs), 1, max(max(d, default=0) for d in depth) + 1), -1)
        kept = []
        for r, n in enumerate(nodes):
            for i in range(n):
                seen = list(range(base[r])) + [base[r] + j for j in range(n) if int(masks[r][i]) >> j & 1]
                for h in range(HQ):
                    self.check(out[start[r] + i, h], q[start[r] + i, h], r, h, seen)
            path, i = [], (n and int(self.rng.integers(0, n))) if n else -1
            while n and i >= 0:
                path.insert(0, i)
                i = parents[r][i]
            keep[r, 0, :len(path)] = path
            kept.append(len(path))
            rows = list(range(base[r])) + [base[r] + j for j in path]
            for g in range(HKV):
                self.k[r][g], self.v[r][g], self.s[r][g] = (x[rows] for x in (self.k[r][g], self.v[r][g], self.s[r][g]))
            self.next_pos[r] += len(path)
        self.ops.compact_kv(self.kc, self.vc, tables, lens, i32(keep), i32(kept), base=i32(base))
        for r, s in enumerate(self.seqs):
            self.alloc.compact(s, base[r], base[r] + kept[r])


@pytest.mark.parametrize("seed,dtype", [(0, torch.bfloat16), (1, torch.float16)])
def test_a_serving_loop(seed, dtype):
    lp = Loop(seed, [3, 8, 5], dtype)
    lengths = [37, 200, 5]
    lp.write([list(range(n)) for n in lengths])
    lp.next_pos = list(lengths)
    for _ in range(3):
        lp.decode()
    used = 60 - lp.alloc.num_free()
    lp.evict(2, 30, 17)
    assert 60 - lp.alloc.num_free() < used          # the long sequence gave blocks back
    for _ in range(2):
        lp.decode()
    lp.tree([5, 17, 1])
    lp.decode()
    lp.tree([33, 2, 9])
    lp.evict(1, 9, 6)
    lp.decode()
    assert lp.ops.get_device_error() == 0
    for r, s in enumerate(lp.seqs):
        assert lp.alloc.seq_len(s) == len(lp.k[r][0]) == len(lp.k[r][1])
        assert lp.alloc.block_table(s) and len(lp.alloc.block_table(s)) == -(-lp.alloc.seq_len(s) // BS)
        lp.alloc.free_seq(s)
    assert lp.alloc.num_free() == 60
