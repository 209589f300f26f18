"""Score-keeping decode, budget selection and in-place compaction
(pa_decode_accumulate, pa_evict_select, pa_compact_kv) against float64 or
index-exact forms.

Tolerance of a score's increase: sum over the group of p (1 + e), with
e <= 2 (D + 4) 2^-24 scale max|q||k| from the scores (numerator and
denominator) and 2^-19 for the exponentials (2 ulp each), the sums of up to
L / 16 terms a lane (each rounding at most 2^-24 of the sum, L <= 4096: 2^-16)
and the divide; then one fp32 rounding of the total, 2^-24 of it.
"""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

DT = {"bf16": torch.bfloat16, "fp16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def built():
    from paged_kv_cache_76_gb300 import _lib
    try:
        _lib.lib()
    except _lib.LibraryMissing:
        from paged_kv_cache_76_gb300 import build
        build.build()
    torch.cuda.init()


def ops():
    from paged_kv_cache_76_gb300 import ops as o
    return o


def cache(seed, lens, hkv, d, bs, dt, extra=1):
    rng = np.random.default_rng(seed)
    nblk = [-(-max(L, 1) // bs) for L in lens]
    nb = sum(nblk) + 3
    perm = rng.permutation(nb)
    tables = np.full((len(lens), max(nblk) + extra), -1, dtype=np.int32)
    off = 0
    for r, n in enumerate(nblk):
        tables[r, :n] = perm[off:off + n]
        off += n
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc = (torch.randn(nb, bs, hkv, d, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    return kc, vc, torch.from_numpy(tables).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"), rng, g


def tokens(c, tables, r, L, bs):
    return c[tables[r, :-(-max(L, 1) // bs)].long()].flatten(0, 1)[:L]


# --------------------------------------------------------------------------- accumulate
ACC = [
    # lens, q_heads, kv_heads, d, bs, dtype, split
    ([700, 1, 0, 1025, 33], 32, 8, 128, 16, "bf16", 0),
    ([2000, 17, 513], 28, 4, 128, 16, "bf16", 256),       # 7 heads a group: odd
    ([300, 40], 16, 1, 64, 4, "fp16", 64),                # 16 heads a group
    ([900, 5], 12, 12, 64, 8, "bf16", 0),                 # one head a group
    ([4000, 100, 3999], 8, 2, 128, 32, "fp16", 128),      # over 30 partitions
]


@pytest.mark.parametrize("case", ACC, ids=[f"h{c[1]}x{c[2]}_d{c[3]}_bs{c[4]}" for c in ACC])
def test_accumulate_matches_float64_and_decode(case):
    lens, hq, hkv, d, bs, dt, split = case
    kc, vc, tables, lens_t, rng, g = cache(1, lens, hkv, d, bs, dt)
    q = (2 * torch.randn(len(lens), hq, d, generator=g, device="cuda")).to(DT[dt])
    width = max(lens) + 37
    rows = torch.from_numpy(rng.permutation(len(lens) + 3)[:len(lens)].astype(np.int32)).cuda()
    scores = torch.rand(len(lens) + 3, hkv, width, generator=g, device="cuda")
    before, scale = scores.clone(), 1 / np.sqrt(d)
    out, into = ops().decode_accumulate(q, kc, vc, tables, lens_t, scale, scores, score_rows=rows, split_tokens=split)
    assert into is scores and ops().get_device_error() == 0
    same = ops().decode_accumulate_split_tokens(len(lens), hq, hkv, tables.shape[1], bs, split)
    assert torch.equal(out, ops().decode(q, kc, vc, tables, lens_t, scale, split_tokens=same))
    apart = torch.full_like(scores, 9.0)
    ops().decode_accumulate(q, kc, vc, tables, lens_t, scale, before, score_rows=rows, scores_out=apart,
                            split_tokens=split)
    for r, L in enumerate(lens):
        row = int(rows[r])
        assert torch.equal(scores[row, :, L:], before[row, :, L:])
        assert bool((apart[row, :, L:] == 9.0).all()) and torch.equal(apart[row, :, :L], scores[row, :, :L])
        if L == 0:
            continue
        k = tokens(kc, tables, r, L, bs).double().repeat_interleave(hq // hkv, 1)
        s = torch.einsum("hd,thd->ht", q[r].double(), k) * scale
        p = torch.softmax(s, 1)
        size = torch.einsum("hd,thd->ht", q[r].double().abs(), k.abs()).amax(1, keepdim=True) * scale
        e = 2 * (d + 4) * 2.0 ** -24 * size + 2.0 ** -16 + 2.0 ** -19
        want = before[row, :, :L].double() + p.view(hkv, -1, L).sum(1)
        tol = (p * e).view(hkv, -1, L).sum(1) + 2.0 ** -23 * want
        assert bool(((scores[row, :, :L].double() - want).abs() <= tol).all())
    others = [i for i in range(scores.shape[0]) if i not in rows.tolist()]
    assert torch.equal(scores[others], before[others]) and bool((apart[others] == 9.0).all())


def test_accumulate_rows_that_are_refused_or_absent():
    from paged_kv_cache_76_gb300 import _lib
    lens = [100, 90, 80, 70]
    kc, vc, tables, lens_t, rng, g = cache(2, lens, 2, 128, 16, "bf16")
    q = torch.randn(4, 8, 128, generator=g, device="cuda").to(torch.bfloat16)
    plain = ops().decode(q, kc, vc, tables, lens_t, 0.1,
                         split_tokens=ops().decode_accumulate_split_tokens(4, 8, 2, tables.shape[1], 16))

    def run(rows, width=128, n=4):
        s = torch.zeros(n, 2, width, device="cuda")
        out, _ = ops().decode_accumulate(q, kc, vc, tables, lens_t, 0.1, s,
                                         score_rows=torch.tensor(rows, dtype=torch.int32, device="cuda"))
        assert torch.equal(out, plain)  # the output does not depend on the rows
        return s, ops().get_device_error()

    good, err = run([0, 1, 2, 3])
    assert err == 0 and torch.equal(ops().decode_accumulate(q, kc, vc, tables, lens_t, 0.1,
                                                            torch.zeros(4, 2, 128, device="cuda"))[1], good)
    s, err = run([0, -1, 2, 3])
    assert err == 0 and torch.count_nonzero(s[1]) == 0 and torch.equal(s[2:], good[2:])
    s, err = run([0, 9, 2, 3])
    assert err == _lib.PA_DEVERR_SCORE_ROW and torch.equal(s[0], good[0]) and torch.count_nonzero(s[1]) == 0
    s, err = run([0, 1, 1, 3])     # the first of two keeps score
    assert err == _lib.PA_DEVERR_SCORE_ROW and torch.equal(s[1], good[1]) and torch.equal(s[3], good[3])
    s, err = run([0, 1, 2, 3], width=96)   # a context longer than the scores
    assert err == _lib.PA_DEVERR_CONTEXT_LEN and torch.equal(s, good[..., :96])


# --------------------------------------------------------------------------- select
def select_reference(scores, lens, rows, sink, heavy, recent):
    hkv, budget = scores.shape[1], sink + heavy + recent
    keep = np.full((len(lens), hkv, budget), -1, dtype=np.int64)
    for r, L in enumerate(lens):
        for g in range(hkv):
            s = scores[rows[r], g, :L].astype(np.float64)
            if L <= budget:
                idx = np.arange(L)
            else:
                mid = np.arange(sink, L - recent)
                v = np.where(np.isnan(s[mid]), -np.inf, s[mid])
                tie = np.isnan(s[mid]).astype(int)
                best = mid[np.lexsort((mid, tie, -v))][:heavy]
                idx = np.sort(np.concatenate([np.arange(sink), best, np.arange(L - recent, L)]))
            keep[r, g, :len(idx)] = idx
    return keep, np.minimum(lens, budget)


SEL = [
    # lens, kv_heads, sink, heavy, recent, kind
    ([1000, 37, 1, 0, 513, 4096], 8, 4, 60, 64, "heavy"),
    ([1000, 37, 999, 20], 2, 0, 16, 0, "ties"),
    ([5000, 5001, 333], 3, 1, 300, 33, "equal"),           # one value only: the lowest indices
    ([70000, 20000, 65537], 2, 4, 8000, 500, "heavy"),
    ([131072], 1, 0, 1, 0, "heavy"),
    ([131071, 4000], 2, 7, 60000, 9, "spread"),
    ([300, 400], 4, 5, 0, 40, "heavy"),                    # nothing by score
    ([300, 257, 258], 4, 0, 256, 1, "special"),
    ([3000, 2999], 4, 0, 100, 0, "negative"),
    ([2000] * 40, 16, 2, 500, 100, "ties"),
]


def make_scores(kind, shape, g):
    x = torch.randn(shape, generator=g, device="cuda")
    if kind == "heavy":
        return x.mul(2).exp()
    if kind == "ties":
        return x.abs().mul(4).round()
    if kind == "equal":
        return torch.full(shape, 0.25, device="cuda")
    if kind == "spread":
        return torch.rand(shape, generator=g, device="cuda")
    if kind == "negative":
        return x
    x = x.clone()
    x[..., ::7], x[..., 3::11], x[..., 5::13] = 0.0, -0.0, float("nan")
    x[..., 6::17], x[..., 9::19] = float("inf"), float("-inf")
    return x


@pytest.mark.parametrize("case", SEL, ids=[f"n{len(c[0])}_L{max(c[0])}_{c[5]}" for c in SEL])
def test_select_is_exact(case):
    lens, hkv, sink, heavy, recent, kind = case
    g = torch.Generator(device="cuda").manual_seed(3)
    rng = np.random.default_rng(3)
    rows = rng.permutation(len(lens) + 2)[:len(lens)].astype(np.int32)
    scores = make_scores(kind, (len(lens) + 2, hkv, max(lens) + 3), g)
    keep, n = ops().evict_select(scores, torch.tensor(lens, dtype=torch.int32, device="cuda"), sink, heavy, recent,
                                 score_rows=torch.from_numpy(rows).cuda())
    assert ops().get_device_error() == 0
    want, wn = select_reference(scores.cpu().numpy(), lens, rows, sink, heavy, recent)
    assert n.tolist() == list(wn)
    assert np.array_equal(keep.cpu().numpy(), want)


def test_select_refuses_bad_rows_and_lengths():
    from paged_kv_cache_76_gb300 import _lib
    s = torch.rand(3, 2, 100, device="cuda")
    i32 = lambda *x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    keep, n = ops().evict_select(s, i32(50, 101, 60), 1, 5, 4)
    assert ops().get_device_error() == _lib.PA_DEVERR_CONTEXT_LEN
    assert n.tolist() == [10, 0, 10] and bool((keep[1] == -1).all())
    keep, n = ops().evict_select(s, i32(50, 50, -2), 1, 5, 4, score_rows=i32(0, 0, 1))   # rows may repeat
    assert ops().get_device_error() == _lib.PA_DEVERR_CONTEXT_LEN
    assert n.tolist() == [10, 10, 0] and torch.equal(keep[0], keep[1])
    keep, n = ops().evict_select(s, i32(50, 50), 1, 5, 4, score_rows=i32(3, -1))
    assert ops().get_device_error() == _lib.PA_DEVERR_SCORE_ROW
    assert n.tolist() == [0, 0] and bool((keep == -1).all())


# --------------------------------------------------------------------------- compact
def compact_reference(kc, vc, tables, lens, keep, n, base, scores, rows, bs):
    kc2, vc2 = kc.clone(), vc.clone()
    s2 = scores.clone() if scores is not None else None
    tb = tables.long()
    for r, L in enumerate(lens):
        b, m = base[r], n[r]
        for h in range(kc.shape[2]):
            src = keep[r, min(h, keep.shape[1] - 1), :m].long() + b
            dst = torch.arange(b, b + m, device="cuda")
            for new, old in ((kc2, kc), (vc2, vc)):
                new[tb[r, dst // bs], dst % bs, h] = old[tb[r, src // bs], src % bs, h]
            if s2 is not None and rows[r] >= 0:
                s2[rows[r], h, b + m:L] = 0
                s2[rows[r], h, b:b + m] = scores[rows[r], h, src]
    return kc2, vc2, s2


COM = [
    # lens, base, keep counts, per head, kv_heads, d, bs, dtype, scores
    ([1000, 37, 500], [0, 0, 0], [256, 37, 499], True, 8, 128, 16, "bf16", True),
    ([300, 40, 64], [290, 30, 1], [5, 10, 0], False, 4, 128, 16, "fp16", False),
    ([700, 1, 5], [0, 0, 2], [700, 1, 2], True, 2, 64, 4, "bf16", True),
    ([5000, 4999], [4, 0], [3000, 2500], True, 3, 64, 8, "fp16", True),
    ([2049, 100], [1, 99], [1025, 1], False, 1, 128, 32, "bf16", True),
    ([20000], [0], [9000], True, 8, 128, 16, "bf16", True),
]


@pytest.mark.parametrize("case", COM, ids=[f"L{max(c[0])}_h{c[4]}_d{c[5]}_bs{c[6]}" for c in COM])
@pytest.mark.parametrize("which", ["random", "late", "early"])
def test_compact_is_exact(case, which):
    lens, base, n, per_head, hkv, d, bs, dt, with_scores = case
    kc, vc, tables, lens_t, rng, g = cache(4, lens, hkv, d, bs, dt)
    heads = hkv if per_head else 1
    keep = np.full((len(lens), heads, max(n) + 2), -1, dtype=np.int32)
    for r in range(len(lens)):
        room = lens[r] - base[r]
        for h in range(heads):
            if which == "random":
                idx = np.sort(rng.permutation(room)[:n[r]])
            elif which == "late":      # the last ones: every move is far
                idx = np.arange(room - n[r], room)
            else:                      # all but one of the first: every move is by one
                idx = np.arange(n[r]) if n[r] == room else np.arange(1, n[r] + 1)
            keep[r, h, :n[r]] = idx
    keep = torch.from_numpy(keep).cuda()
    rows = rng.permutation(len(lens) + 1)[:len(lens)].astype(np.int32)
    scores = torch.rand(len(lens) + 1, hkv, max(lens) + 5, generator=g, device="cuda") if with_scores else None
    want = compact_reference(kc, vc, tables, lens, keep, n, base, scores, rows, bs)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    ops().compact_kv(kc, vc, tables, lens_t, keep, i32(n), base=i32(base) if any(base) else None, scores=scores,
                     score_rows=torch.from_numpy(rows).cuda() if with_scores else None)
    assert ops().get_device_error() == 0
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1])
    if with_scores:
        assert torch.equal(scores, want[2])


def test_compact_refuses_what_it_cannot_do():
    from paged_kv_cache_76_gb300 import _lib
    kc, vc, tables, lens_t, rng, g = cache(5, [100, 90], 2, 128, 16, "bf16")
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")  # noqa: E731
    k0, v0 = kc.clone(), vc.clone()

    def run(keep, n, code, lens=lens_t, base=None, tables=tables, scores=None, score_rows=None):
        kc.copy_(k0), vc.copy_(v0)
        ops().compact_kv(kc, vc, tables, lens, i32(keep), i32(n), base=base, scores=scores, score_rows=score_rows)
        assert ops().get_device_error() == code

    run([[[3, 5, 9]], [[1, 2, 3]]], [3, 4], _lib.PA_DEVERR_KEEP)          # more than the list holds: request 1 stays
    assert torch.equal(tokens(kc, tables, 1, 90, 16), tokens(k0, tables, 1, 90, 16))
    assert torch.equal(tokens(kc, tables, 0, 100, 16)[:3], tokens(k0, tables, 0, 100, 16)[[3, 5, 9]])
    run([[[3, 0, 100]], [[1, 2, 3]]], [3, 3], _lib.PA_DEVERR_KEEP)        # a source before its place; one past the end
    got, old = tokens(kc, tables, 0, 100, 16), tokens(k0, tables, 0, 100, 16)
    assert torch.equal(got[0], old[3]) and torch.equal(got[1:], old[1:])
    run([[[3, 5, 9]], [[1, 2, 3]]], [3, 3], _lib.PA_DEVERR_KEEP, base=i32([98, 0]))      # base + count > L
    assert torch.equal(tokens(kc, tables, 0, 100, 16), old)
    run([[[3, 5, 9]], [[1, 2, 3]]], [3, 3], _lib.PA_DEVERR_CONTEXT_LEN, lens=i32([100, 9000]))
    bad = tables.clone()
    bad[0, 0] = -5
    run([[[20, 21, 22]], [[1, 2, 3]]], [3, 3], _lib.PA_DEVERR_BLOCK_ID, tables=bad)
    assert torch.equal(kc[tables[0].clamp_min(0).long()], k0[tables[0].clamp_min(0).long()])
    s = torch.rand(2, 2, 100, generator=g, device="cuda")
    s0 = s.clone()
    run([[[3, 5, 9]], [[1, 2, 3]]], [3, 3], _lib.PA_DEVERR_SCORE_ROW, scores=s, score_rows=i32([1, 1]))
    assert torch.equal(s[0], s0[0]) and torch.equal(s[1, :, :3], s0[1][:, [3, 5, 9]])
    assert torch.count_nonzero(s[1, :, 3:]) == 0


def test_streams_graphs_and_recordings():
    lens = [600, 70, 2000]
    kc, vc, tables, lens_t, rng, g = cache(6, lens, 4, 128, 16, "bf16")
    q = torch.randn(3, 16, 128, generator=g, device="cuda").to(torch.bfloat16)
    s = torch.rand(3, 4, 2000, generator=g, device="cuda")
    k0, v0 = kc.clone(), vc.clone()

    def step():
        into = torch.empty_like(s).copy_(s)
        out, _ = ops().decode_accumulate(q, kc, vc, tables, lens_t, 0.09, into)
        keep, n = ops().evict_select(into, lens_t, 4, 60, 36)
        ops().compact_kv(kc, vc, tables, lens_t, keep, n, scores=into)
        return out, into, keep, n

    def restore():
        kc.copy_(k0), vc.copy_(v0)

    want = [x.clone() for x in step()] + [kc.clone(), vc.clone()]
    restore()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = step()
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(want, list(got) + [kc, vc]))
    restore()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = step()
    restore()
    graph.replay()
    assert all(torch.equal(a, b) for a, b in zip(want, list(got) + [kc, vc]))
    assert ops().get_device_error() == 0
