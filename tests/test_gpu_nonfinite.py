"""Infinities and NaN in the operators over moved caches: they decide exactly
the results that the formulas give them, and no others."""
import numpy as np
import pytest
import torch

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


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


def i32(*x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def same(a, b):
    """The same bits, any NaN equal to any other."""
    bits = torch.int16 if a.element_size() == 2 else torch.int32
    return bool(((a.view(bits) == b.view(bits)) | (a.isnan() & b.isnan())).all())


@pytest.mark.parametrize("norm", [False, True])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,dtype", [(128, 64, torch.bfloat16), (128, 16, torch.float16), (64, 48, torch.bfloat16)])
def test_elements_that_are_not_rotated_stay_apart(d, rot, dtype, interleaved, norm):
    """Behind rot_dim an element meets no other one: an infinity or a NaN there stays where it is (with a norm, the
    row's infinite or NaN factor makes the finite ones 0 or NaN, by the formula); in a rotated pair it stays in it."""
    g = torch.Generator(device="cuda").manual_seed(11)
    T, hq, hkv, bs = 13, 5, 2, 16
    q, k, v = (torch.randn(T, h, d, generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    for x in (q, k):
        x[0, 0, rot], x[1, 1, rot + 5], x[2, 0, d - 1], x[3, 1, rot + 3] = INF, -INF, NAN, -0.0
        x[4, 0, 3], x[5, 1, rot // 2 + 1] = INF, NAN   # in a pair
    pos, slots = torch.arange(T, dtype=torch.int32, device="cuda") + 1, torch.arange(T, dtype=torch.int32, device="cuda")
    table = ops().rope_table(50, rot, device="cuda")
    kc, vc = (torch.zeros(2, bs, hkv, d, dtype=dtype, device="cuda") for _ in range(2))
    w = torch.ones(d, dtype=dtype, device="cuda") if norm else None
    out = ops().norm_rope_and_cache(q, k, v, pos, table, slots, kc, vc, q_weight=w, k_weight=w, interleaved=interleaved)
    assert ops().get_device_error() == 0
    lo, hi = (np.arange(0, rot, 2), np.arange(1, rot, 2)) if interleaved else (np.arange(rot // 2),
                                                                                np.arange(rot // 2, rot))
    c, s = table[pos.long(), None, :rot // 2], table[pos.long(), None, rot // 2:]
    for x, got in ((q, out), (k, kc.flatten(0, 1)[:T])):
        y = x.float()
        if norm:
            y = y * torch.rsqrt((y * y).mean(-1, keepdim=True) + 1e-6)
        z = y.clone()
        z[..., lo], z[..., hi] = y[..., lo] * c - y[..., hi] * s, y[..., hi] * c + y[..., lo] * s
        assert torch.equal(got.isnan(), z.isnan()) and torch.equal(got.isinf(), z.isinf())
        assert torch.equal(got[got.isinf()].float(), z[z.isinf()])
        if not norm:
            assert same(got[..., rot:], x[..., rot:])


@pytest.mark.parametrize("nodes,hq,hkv,bs,split", [(40, 8, 2, 16, 0), (64, 12, 3, 4, 256), (33, 16, 2, 8, 128)])
def test_every_row_of_both_tiles_learns_of_a_value(nodes, hq, hkv, bs, split):
    """More than 128 rows per KV head, which two groups of warps share: each row is non-finite in a dimension exactly
    where a node that it sees is, whichever group met the value first."""
    d, reqs = 64, 24
    rng = np.random.default_rng(14)
    g = torch.Generator(device="cuda").manual_seed(14)
    lens = [int(x) + nodes for x in rng.integers(0, 400, reqs)]
    blocks = -(-max(lens) // bs)
    tables = torch.arange(reqs * blocks, dtype=torch.int32, device="cuda").view(reqs, blocks)
    kc, vc = (torch.randn(reqs * blocks, bs, hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(reqs * nodes, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    trees = [[int(rng.integers(max(-1, i - 4), i)) for i in range(nodes)] for _ in range(reqs)]
    mask = torch.cat([ops().tree_mask(t) for t in trees]).cuda()
    v = vc.view(reqs, blocks * bs, hkv, d)
    bad = torch.zeros(reqs, nodes, d, dtype=torch.bool)
    for r, L in enumerate(lens):
        for j in rng.permutation(nodes)[:5]:
            e = int(rng.integers(d))
            v[r, L - nodes + int(j), :, e] = (INF, -INF, NAN)[int(rng.integers(3))]
            bad[r, int(j), e] = True
    sees = (mask.view(reqs, nodes, 1).cpu() >> torch.arange(nodes)) & 1
    want = torch.einsum("rij,rje->rie", sees.float(), bad.float()) > 0
    for _ in range(10):
        out = ops().verify_tree(q, i32(*range(0, reqs * nodes + 1, nodes)), mask, i32(*lens), kc, vc, tables, d ** -0.5,
                                nodes, split_tokens=split)
        assert ops().get_device_error() == 0
        got = ~out.isfinite().cpu().view(reqs, nodes, hq, d)
        assert torch.equal(got, want[:, :, None].expand_as(got))


@pytest.mark.parametrize("hq,hkv,split", [(8, 2, 0), (8, 2, 64), (14, 2, 0), (2, 2, 64)])
def test_scores_of_a_softmax_that_is_not_a_number(hq, hkv, split):
    """A NaN or a positively infinite logit makes its head's weights NaN for every token of the request, and so the
    scores of its KV head; a negatively infinite one weighs nothing.  No other score changes."""
    lens, d, bs = [300, 70, 1, 200], 128, 16
    g = torch.Generator(device="cuda").manual_seed(12)
    tables = torch.arange(4 * 20, dtype=torch.int32, device="cuda").view(4, 20)
    kc, vc = (torch.randn(80, bs, hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    q = torch.randn(4, hq, d, generator=g, device="cuda").to(torch.bfloat16)
    clean = torch.rand(4, hkv, 320, generator=g, device="cuda")
    before = clean.clone()
    ops().decode_accumulate(q, kc, vc, tables, i32(*lens), 0.09, clean, split_tokens=split)
    keys = kc.view(4, 320, hkv, d)
    keys[0, 299, 1, 7] = NAN         # one token of the last partition
    keys[1, :, 0] = NAN              # every token
    keys[2, 0, 0, 3] = NAN           # the only token
    keys[3, 5, 0, 9] = INF           # by the sign of the query: a NaN, or a weight of nothing
    got = before.clone()
    ops().decode_accumulate(q, kc, vc, tables, i32(*lens), 0.09, got, split_tokens=split)
    assert ops().get_device_error() == 0
    for r, L in enumerate(lens):
        k = keys[r, :L].double().repeat_interleave(hq // hkv, 1)
        p = torch.softmax(torch.einsum("hd,thd->ht", q[r].double(), k) * 0.09, 1)
        want = before[r, :, :L].double() + p.view(hkv, -1, L).sum(1)
        assert torch.equal(got[r, :, :L].isnan(), want.isnan()), r
        fine = ~want.isnan()
        assert bool(((got[r, :, :L].double() - want)[fine].abs() < 1e-4).all())
        assert torch.equal(got[r, :, L:], before[r, :, L:])
    assert torch.equal(got[0, 0], clean[0, 0]) and torch.equal(got[1, 1], clean[1, 1])
    assert torch.equal(got[2, 1], clean[2, 1]) and torch.equal(got[3, 1], clean[3, 1])


@pytest.mark.parametrize("nodes,hq,bs", [(7, 8, 16), (30, 16, 16), (64, 16, 16), (64, 16, 4)])
def test_a_seen_value_decides_however_small_its_weight(nodes, hq, bs):
    """A key of the first partition takes all the weight that 32 bits can hold, and a drafted node in the last one has
    an infinity and a NaN among its values: the rows that see the node are infinite and NaN there, cut or whole."""
    hkv, d, hist = 2, 128, 700
    g = torch.Generator(device="cuda").manual_seed(13)
    L = hist + nodes
    nb = -(-L // bs)
    tables = torch.arange(nb, dtype=torch.int32, device="cuda")[None]
    kc, vc = (torch.randn(nb, bs, hkv, d, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    along = torch.randn(d, generator=g, device="cuda").sign()
    q = (along + 0.1 * torch.randn(nodes, hq, d, generator=g, device="cuda")).to(torch.bfloat16)
    kc.view(-1, hkv, d)[3] = (30 * along).to(torch.bfloat16)     # logits of about 30 d / sqrt(d) = 340
    mask = ops().tree_mask([-1] + [max(0, i - 3) if i != 2 else -1 for i in range(1, nodes)]).cuda()
    args = (q, i32(0, nodes), mask, i32(L), kc, vc, tables, d ** -0.5, nodes)
    clean = ops().verify_tree(*args, split_tokens=128)
    v = vc.view(-1, hkv, d)
    v[hist + 1, :, 5], v[hist + 1, :, 6], v[hist + 1, :, 7] = INF, NAN, -INF
    seen = torch.tensor([bool((int(m) >> 1) & 1) for m in mask], device="cuda")
    assert 0 < int(seen.sum()) < nodes
    for split in (128, 256, -(-(nb * bs) // 128) * 128):
        got = ops().verify_tree(*args, split_tokens=split)
        assert ops().get_device_error() == 0
        assert torch.equal(got[seen][..., 5], torch.full_like(got[seen][..., 5], INF))
        assert torch.equal(got[seen][..., 7], torch.full_like(got[seen][..., 7], -INF))
        assert bool(got[seen][..., 6].isnan().all())
        rest = [i for i in range(d) if i not in (5, 6, 7)]
        assert bool(got[~seen].isfinite().all()) and bool(got[..., rest].isfinite().all())
        if split == 128:
            assert torch.equal(got[~seen], clean[~seen]) and torch.equal(got[..., rest], clean[..., rest])
