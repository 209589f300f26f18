"""The forms of the score-keeping decode, the selection and the compaction that
large batches and long contexts take: merges by whole CTAs, every padded group
size, rows held in shared memory in part, and the compaction's three pipelines.
Each case states the rule that leads to its form, so that it cannot slip into
another one.

Tolerance of a score's increase: as in test_gpu_eviction.py, with the number of
sums as it is here.  A lane adds at most L / 16 probabilities in all, then 3
lanes' sums; the second pass at most ceil(partitions / 32) + 4 products and
sums of a lane, then 5 lanes' sums, an inverse and a product: for at most 512
partitions under L / 16 + 64 roundings of 2^-24.
"""
import numpy as np
import pytest
import torch

from test_gpu_eviction import built, cache, compact_reference, make_scores, ops, select_reference, tokens  # noqa: F401

pytestmark = pytest.mark.gpu


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32).cuda()


def sms():
    return torch.cuda.get_device_properties(0).multi_processor_count


ACC = [
    # lens, q_heads, kv_heads, d, bs, dtype, split, partitions
    ([9000, 2100, 65], 8, 4, 128, 16, "bf16", 64, 141),       # 2 heads a group; several rounds of a lane's partitions
    ([2072, 100, 0], 20, 2, 64, 16, "fp16", 64, 33),          # 10 heads; one partition more than a warp merges
    ([40000, 3], 4, 2, 64, 32, "bf16", 256, 157),
    ([9000, 8999], 12, 1, 128, 16, "fp16", 64, 141),          # 12 heads
    ([20000, 700], 14, 2, 128, 4, "bf16", 128, 157),          # 7 heads
    ([5000, 16], 16, 1, 128, 8, "bf16", 64, 79),
    ([5000, 16], 3, 3, 64, 8, "fp16", 64, 79),
    ([700, 40, 1], 20, 2, 128, 16, "bf16", 64, 12),           # merged by warps: groups of 10, 2 and 3
    ([700, 40, 1], 4, 2, 64, 8, "fp16", 64, 12),
    ([700, 40, 1], 6, 2, 128, 32, "bf16", 64, 12),
]


@pytest.mark.parametrize("case", ACC, ids=[f"h{c[1]}x{c[2]}_d{c[3]}_bs{c[4]}_p{c[7]}" for c in ACC])
def test_accumulate_over_many_partitions(case):
    lens, hq, hkv, d, bs, dt, split, parts = case
    kc, vc, tables, lens_t, rng, g = cache(21, lens, hkv, d, bs, dt)
    assert -(-tables.shape[1] * bs // split) == parts     # the CTA's merge from 33 on
    q = (2 * torch.randn(len(lens), hq, d, generator=g, device="cuda")).to(kc.dtype)
    rows = i32(rng.permutation(len(lens) + 2)[:len(lens)])
    scores = torch.rand(len(lens) + 2, hkv, max(lens) + 9, generator=g, device="cuda")
    before, scale = scores.clone(), 1 / np.sqrt(d)
    out, _ = ops().decode_accumulate(q, kc, vc, tables, lens_t, scale, scores, score_rows=rows, split_tokens=split)
    assert ops().get_device_error() == 0
    assert torch.equal(out, ops().decode(q, kc, vc, tables, lens_t, scale, split_tokens=split))
    again = before.clone()
    ops().decode_accumulate(q, kc, vc, tables, lens_t, scale, again, score_rows=rows, split_tokens=split)
    assert torch.equal(again, scores)
    for r, L in enumerate(lens):
        row = int(rows[r])
        assert torch.equal(scores[row, :, L:], before[row, :, L:])
        if L == 0:
            continue
        k = tokens(kc, tables, r, L, bs).double().repeat_interleave(hq // hkv, 1)
        p = torch.softmax(torch.einsum("hd,thd->ht", q[r].double(), k) * scale, 1)
        size = torch.einsum("hd,thd->ht", q[r].double().abs(), k.abs()).amax(1, keepdim=True) * scale
        e = 2 * (d + 4) * 2.0 ** -24 * size + (L / 16 + 64) * 2.0 ** -24 + 2.0 ** -19
        want = before[row, :, :L].double() + p.view(hkv, -1, L).sum(1)
        tol = (p * e).view(hkv, -1, L).sum(1) + 2.0 ** -23 * want
        assert bool(((scores[row, :, :L].double() - want).abs() <= tol).all()), r
    others = [i for i in range(len(lens) + 2) if i not in rows.tolist()]
    assert torch.equal(scores[others], before[others])


SEL = [
    # lens, kv_heads, sink, heavy, recent, kind, most CTAs of a row
    ([20000, 19999, 12345, 8193] * 7 + [300], 7, 4, 2000, 64, "heavy", 1),     # more rows than SMs, long ones
    ([20000, 3000] * 14, 7, 0, 5000, 0, "ties", 1),
    ([131009, 65000, 32768, 131008, 50001, 9000, 600, 131007], 8, 4, 4092, 4096, "heavy", 2),   # clusters of 2
    ([131009, 131009, 2000, 40000, 131009, 70000, 131009, 1], 8, 0, 3000, 17, "special", 2),
    ([131072, 100000, 7000], 6, 3, 60000, 1, "spread", 8),
]


@pytest.mark.parametrize("case", SEL, ids=[f"n{len(c[0])}_L{max(c[0])}_{c[5]}" for c in SEL])
def test_select_where_keys_do_not_all_fit(case):
    lens, hkv, sink, heavy, recent, kind, ctas = case
    rows, length = len(lens) * hkv, max(lens) + 3
    assert (rows > sms()) if ctas == 1 else (rows * ctas <= sms() and (ctas == 8 or rows * ctas * 2 > sms()))
    assert length / ctas > 8192        # CTAs of 1024 threads: alone on an SM one holds 40960 keys, two 16384 each
    g = torch.Generator(device="cuda").manual_seed(22)
    scores = make_scores(kind, (len(lens), hkv, length), g)
    keep, n = ops().evict_select(scores, i32(lens), sink, heavy, recent)
    assert ops().get_device_error() == 0
    want, wn = select_reference(scores.cpu().numpy(), lens, range(len(lens)), sink, heavy, recent)
    assert n.tolist() == list(wn)
    assert np.array_equal(keep.cpu().numpy(), want)


COM = [
    # requests, longest context, kv_heads, d, bs, dtype, one list per head, form
    (8, 3000, 8, 128, 16, "bf16", True, 512),
    (8, 2500, 8, 128, 4, "fp16", False, 512),
    (16, 900, 8, 128, 16, "fp16", True, 256),
    (16, 1500, 8, 128, 32, "bf16", False, 256),
    (16, 1200, 8, 64, 8, "bf16", True, 512),
    (40, 700, 8, 64, 16, "fp16", True, 256),
]


@pytest.mark.parametrize("case", COM, ids=[f"n{c[0]}_d{c[3]}_bs{c[4]}_{c[7]}" for c in COM])
@pytest.mark.parametrize("which", ["random", "late", "early"])
def test_compact_of_large_batches_is_exact(case, which):
    reqs, longest, hkv, d, bs, dt, per_head, form = case
    ctas = d // 8 // 4 * hkv * reqs                   # of 64-byte columns
    assert (sms() < ctas <= 2 * sms()) if form == 512 else ctas > 2 * sms()
    rng = np.random.default_rng(23)
    lens = [longest, longest - 1, 70] + rng.integers(1, longest, reqs - 3).tolist()
    base = [int(rng.integers(0, L // 2 + 1)) for L in lens]
    n = [int(rng.integers(0, L - b + 1)) for L, b in zip(lens, base)]
    base[0], n[0], n[1] = 0, longest - 7, 0
    kc, vc, tables, lens_t, _, g = cache(23, lens, hkv, d, bs, dt)
    heads = hkv if per_head else 1
    keep = np.full((reqs, heads, max(n) + 3), -1, dtype=np.int32)
    assert keep.shape[2] > 64                         # not the one-step kernel's
    for r in range(reqs):
        room = lens[r] - base[r]
        for h in range(heads):
            if which == "random":
                idx = np.sort(rng.permutation(room)[:n[r]])
            elif which == "late":
                idx = np.arange(room - n[r], room)
            else:
                idx = np.arange(n[r]) if n[r] == room else np.arange(1, n[r] + 1)
            keep[r, h, :n[r]] = idx
    keep = torch.from_numpy(keep).cuda()
    rows = rng.permutation(reqs + 1)[:reqs].astype(np.int32)
    scores = torch.rand(reqs + 1, hkv, longest + 5, generator=g, device="cuda")
    want = compact_reference(kc, vc, tables, lens, keep, n, base, scores, rows, bs)
    ops().compact_kv(kc, vc, tables, lens_t, keep, i32(n), base=i32(base), scores=scores, score_rows=i32(rows))
    assert ops().get_device_error() == 0
    assert torch.equal(kc, want[0]) and torch.equal(vc, want[1]) and torch.equal(scores, want[2])
