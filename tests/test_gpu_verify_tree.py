"""Attention of drafted trees (pa_verify_tree) against a float64 form, over
tree sizes 1 to 64, group sizes, block sizes, ragged batches, split contexts,
rows that see nothing, and non-finite values in places that are not seen.

Tolerance, per element, with u = eps/2 of the type, p the exact weights and
A = sum_t p_t |v_t|: each weight is rounded to the type for the P.V product
(relative u), the denominator sums either the rounded or the unrounded weights
(another u on the result at most), and the output is rounded once (u |ref|):
2 u |ref| + u A together, plus the fp32 part: the error of a score is at most
(D + 4) 2^-24 scale sum_d |q_d k_d|, which moves a weight by that relative
amount (twice: numerator and denominator), and 2^-20 A covers the exponentials
(2^-22 relative each) and the sums.
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


def make(seed, hist, nodes, hq, hkv, d, bs, dt, extra=2):
    """Requests with hist[r] context tokens and nodes[r] drafted ones, random trees."""
    rng = np.random.default_rng(seed)
    lens = [a + b for a, b in zip(hist, nodes)]
    nblk = [max(-(-L // bs), 1) for L in lens]
    nb = sum(nblk) + 5
    perm = rng.permutation(nb)
    tables = np.full((len(lens), max(nblk) + extra), -1, dtype=np.int32)
    off = 0
    for r, n in enumerate(nblk):
        tables[r, :n] = perm[off:off + n]
        off += n
    masks = []
    for n in nodes:
        parents = [int(rng.integers(max(-1, i - 5), i)) if i else -1 for i in range(n)]
        masks.append(ops().tree_mask(parents))
    g = torch.Generator(device="cuda").manual_seed(seed)
    kc, vc = (torch.randn(nb, bs, hkv, d, generator=g, device="cuda").to(DT[dt]) for _ in range(2))
    q = (1.5 * torch.randn(sum(nodes), hq, d, generator=g, device="cuda")).to(DT[dt])
    return dict(q=q, q_start=torch.from_numpy(np.concatenate([[0], np.cumsum(nodes)]).astype(np.int32)).cuda(),
                mask=torch.cat(masks).cuda() if masks else torch.zeros(0, dtype=torch.int64, device="cuda"),
                lens=torch.tensor(lens, dtype=torch.int32, device="cuda"), kc=kc, vc=vc,
                tables=torch.from_numpy(tables).cuda(), scale=1 / np.sqrt(d), max_q=max(max(nodes), 1))


def call(c, **kw):
    return ops().verify_tree(c["q"], c["q_start"], c["mask"], c["lens"], c["kc"], c["vc"], c["tables"], c["scale"],
                             c["max_q"], **kw)


def reference(c, r):
    """float64 rows of request r, the mean |v| of each row's weights, and the score error bound per row."""
    qs = c["q_start"].tolist()
    n, L = qs[r + 1] - qs[r], int(c["lens"][r])
    bs, hkv, d = c["kc"].shape[1:]
    ids = c["tables"][r, :-(-L // bs)].long()
    k, v = (x[ids].flatten(0, 1)[:L].double() for x in (c["kc"], c["vc"]))
    q = c["q"][qs[r]:qs[r + 1]].double()
    G = q.shape[1] // hkv
    mask = c["mask"][qs[r]:qs[r + 1]].tolist()
    see = torch.ones(n, L, dtype=torch.bool, device="cuda")
    for i in range(n):
        for j in range(n):
            see[i, L - n + j] = bool((mask[i] >> j) & 1)
    out, mean, err = torch.zeros_like(q), torch.zeros_like(q), torch.zeros(n, q.shape[1], 1, device="cuda").double()
    for h in range(q.shape[1]):
        for i in range(n):
            t = see[i].nonzero().squeeze(1)
            if not len(t):
                continue
            kk, vv = k[t, h // G], v[t, h // G]
            s = kk @ q[i, h] * c["scale"]
            p = torch.softmax(s, 0)
            out[i, h], mean[i, h] = p @ vv, p @ vv.abs()
            err[i, h] = (d + 4) * 2.0 ** -24 * c["scale"] * float((kk.abs() @ q[i, h].abs()).max())
    return out, mean, err


def assert_request(c, got, r, what=""):
    qs = c["q_start"].tolist()
    out, mean, err = reference(c, r)
    u = torch.finfo(got.dtype).eps / 2
    tol = 2 * u * out.abs() + (u + 2 * err + 2.0 ** -20) * mean + 1e-7
    g = got[qs[r]:qs[r + 1]].double()
    assert bool(torch.isfinite(g).all()), f"{what}: request {r} holds non-finite values"
    over = (g - out).abs() - tol
    assert bool((over <= 0).all()), f"{what}: request {r} is {float(over.max())} past its tolerance"


CASES = [
    # hist, nodes, q_heads, kv_heads, d, bs, dtype, split_tokens
    ([700, 0, 33, 1025], [5, 9, 1, 17], 32, 8, 128, 16, "bf16", 0),
    ([300, 64, 127, 128], [64, 63, 64, 33], 8, 2, 128, 16, "bf16", 0),        # up to 256 rows, tails across tiles
    ([2000, 9, 517], [26, 60, 40], 28, 4, 128, 16, "bf16", 512),              # 7 heads a group, split
    ([1500, 640, 639, 641], [3, 8, 1, 64], 16, 1, 128, 32, "fp16", 128),       # 1024 rows of one head
    ([50, 0, 0, 7], [4, 3, 1, 2], 4, 4, 64, 4, "fp16", 0),                     # blocks of 4
    ([1000, 5, 260], [64, 64, 31], 12, 2, 64, 8, "bf16", 256),
    ([0, 0, 3], [64, 1, 2], 6, 2, 64, 16, "fp16", 0),                          # no context before the draft
    ([1, 2, 3, 4, 5, 6, 7, 8], [1] * 8, 8, 8, 128, 16, "bf16", 0),
    ([120, 121, 122, 123], [8, 8, 8, 8], 32, 8, 128, 16, "bf16", 128),         # drafts across a partition's end
    ([5000, 1], [20, 2], 8, 1, 128, 16, "bf16", 0),                            # few requests, automatic split
    ([260, 700], [30, 64], 9, 3, 64, 4, "bf16", 128),
]


@pytest.mark.parametrize("case", CASES, ids=[f"h{c[2]}x{c[3]}_d{c[4]}_bs{c[5]}_{c[6]}_s{c[7]}_{i}"
                                             for i, c in enumerate(CASES)])
def test_matches_float64(case):
    c = make(1, *case[:7])
    got = call(c, split_tokens=case[7])
    assert ops().get_device_error() == 0
    for r in range(len(case[0])):
        assert_request(c, got, r, str(case))
    assert torch.equal(got, call(c, split_tokens=case[7]))  # the same bits again


@pytest.mark.parametrize("nodes", [1, 4, 8])
def test_a_chain_is_the_linear_verify(nodes):
    """A tree whose node j sees nodes 0..j, against verify_decode (each within its rounding of the exact result)."""
    c = make(2, [300, 40, 1000], [nodes] * 3, 16, 4, 128, 16, "bf16")
    c["mask"] = ops().tree_mask([i - 1 for i in range(nodes)]).repeat(3).cuda()
    got = call(c)
    lin = ops().verify_decode(c["q"].view(3, nodes, 16, 128), c["kc"], c["vc"], c["tables"], c["lens"], c["scale"])
    for r in range(3):
        assert_request(c, got, r)
        assert_request(c, lin.reshape(got.shape), r)


def test_rows_that_see_nothing_and_bits_behind_the_tree():
    c = make(3, [0, 200, 0], [6, 6, 64], 8, 2, 128, 16, "bf16")
    m = c["mask"].clone()
    m[2] = 0                       # no context, no node: zeros
    m[8] = 0                       # the context alone
    m[0] |= ~0 << 6                # bits behind the request's nodes: ignored
    c["mask"] = m
    got = call(c)
    assert torch.count_nonzero(got[2]) == 0
    c["mask"] = m.clone()
    c["mask"][0] &= 63
    for r in range(3):
        assert_request(c, got, r)
    assert ops().get_device_error() == 0


@pytest.mark.parametrize("bs,dt,nodes,split", [(16, "bf16", 9, 0), (16, "fp16", 64, 128), (4, "fp16", 9, 0),
                                               (8, "bf16", 33, 128)])
def test_what_a_row_does_not_see_does_not_reach_it(bs, dt, nodes, split):
    """Stale slots behind the context and a padding node hold NaN and infinities; so does one branch of the tree."""
    c = make(4, [250, 121, 60], [nodes] * 3, 16, 4, 128, bs, dt)
    for i in range(3):  # node n-1 is padding: nobody sees it, it sees the context
        c["mask"][nodes * i:nodes * (i + 1)] &= (1 << (nodes - 1)) - 1
    clean = call(c, split_tokens=split)
    for r in range(3):
        assert_request(c, clean, r)
    kc, vc = c["kc"].clone(), c["vc"].clone()

    def slot(r, t):
        return int(c["tables"][r, t // bs]), t % bs

    L = [int(x) for x in c["lens"]]
    for r, bad in ((0, float("nan")), (1, float("inf")), (2, float("-inf"))):
        b, o = slot(r, L[r] - 1)
        kc[b, o], vc[b, o] = bad, bad
        for t in range(L[r], -(-L[r] // bs) * bs):
            b, o = slot(r, t)
            kc[b, o], vc[b, o] = bad, bad
    c["kc"], c["vc"] = kc, vc
    assert torch.equal(call(c, split_tokens=split), clean)
    # node 1 of request 1 holds an infinity in dimension 5 and a NaN in 6 of V: the rows that see it, and no other
    b, o = slot(1, L[1] - nodes + 1)
    vc[b, o, :, 5], vc[b, o, :, 6] = float("inf"), float("nan")
    got = call(c, split_tokens=split)
    seen = torch.tensor([bool((int(m) >> 1) & 1) for m in c["mask"][nodes:2 * nodes]], device="cuda")
    mine = got[nodes:2 * nodes]
    assert bool(torch.isinf(mine[seen][..., 5]).all()) and bool(torch.isnan(mine[seen][..., 6]).all())
    other = torch.ones(128, dtype=torch.bool, device="cuda")
    other[5:7] = False
    assert torch.equal(mine[~seen], clean[nodes:2 * nodes][~seen])
    assert torch.equal(mine[..., other], clean[nodes:2 * nodes][..., other])
    assert torch.equal(got[:nodes], clean[:nodes]) and torch.equal(got[2 * nodes:], clean[2 * nodes:])


def test_refused_requests_and_rows_behind_the_last():
    from paged_kv_cache_76_gb300 import _lib
    c = make(5, [100, 200, 300], [4, 5, 6], 8, 2, 128, 16, "bf16")
    good = call(c)
    lens = c["lens"].clone()

    def run(code, **kw):
        out = torch.full_like(c["q"], 7.0)
        call({**c, **kw}, out=out)
        assert ops().get_device_error() == code
        return out

    short = lens.clone()
    short[1] = 3                                             # shorter than its draft
    out = run(_lib.PA_DEVERR_QUERY_RANGE, lens=short)
    assert bool((out[4:9] == 7.0).all()) and torch.equal(out[:4], good[:4]) and torch.equal(out[9:], good[9:])
    long = lens.clone()
    long[1] = c["tables"].shape[1] * 16 + 1                  # past the table
    out = run(_lib.PA_DEVERR_CONTEXT_LEN, lens=long)
    assert bool((out[4:9] == 7.0).all()) and torch.equal(out[:4], good[:4])
    starts = c["q_start"].clone()
    starts[3] = 40                                           # past total_q
    out = run(_lib.PA_DEVERR_QUERY_RANGE, q_start=starts)
    assert torch.equal(out[:9], good[:9]) and bool((out[9:] == 7.0).all())
    out = run(_lib.PA_DEVERR_QUERY_RANGE, max_q=5)           # six nodes, at most five announced
    assert torch.equal(out[:9], good[:9]) and bool((out[9:] == 7.0).all())
    starts = c["q_start"].clone()
    starts[3] = 14                                           # the last row belongs to nobody
    lens2 = lens.clone()
    lens2[2] -= 1
    out = run(0, q_start=starts, lens=lens2)
    assert bool((out[14:] == 7.0).all()) and torch.equal(out[:9], good[:9])
    starts = c["q_start"].clone()
    starts[1] = 0                                            # a request without rows
    lens3 = lens.clone()
    lens3[1] += 0
    out = run(_lib.PA_DEVERR_NONE, q_start=torch.tensor([0, 4, 4, 10], dtype=torch.int32, device="cuda"),
              lens=torch.tensor([104, 0, 306], dtype=torch.int32, device="cuda"),
              tables=c["tables"])
    assert torch.equal(out[:4], good[:4])
    bad = c["tables"].clone()
    bad[0, 2] = c["kc"].shape[0]
    out = run(_lib.PA_DEVERR_BLOCK_ID, tables=bad)
    assert torch.equal(out[4:], good[4:])


def test_streams_graphs_and_recordings():
    c = make(6, [900, 40, 333], [7, 30, 64], 32, 8, 128, 16, "bf16")
    want = call(c, split_tokens=256)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        got = call(c, split_tokens=256)
    side.synchronize()
    assert torch.equal(got, want)
    g1, g2 = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
    with torch.cuda.graph(g1):
        a = call(c, split_tokens=256)
    with torch.cuda.graph(g2):
        b = call(c, split_tokens=128)
    a.zero_(), b.zero_()
    for g in (g2, g1, g2, g1):
        g.replay()
    assert torch.equal(a, want) and torch.equal(b, call(c, split_tokens=128))
    with ops().recording() as rec:
        got = call(c, split_tokens=256)
    got.zero_()
    rec()
    assert torch.equal(got, want)


@pytest.mark.parametrize("nreq,max_n,bs", [(170, 9, 16), (130, 64, 16), (300, 20, 4)])
def test_a_batch_of_many_lengths(nreq, max_n, bs):
    """More units than the GPU runs at once, which then start in order of
    length, 128 requests at a time: equal lengths, requests without queries or
    context and refused ones, on both sides of the 128.  The order decides when
    a unit runs, never what it computes: every request's rows are bit-identical
    to the request's alone."""
    from paged_kv_cache_76_gb300 import _lib
    g = np.random.default_rng(41 + nreq)
    nodes = g.integers(0, max_n + 1, nreq)
    hist = np.where(g.integers(0, 3, nreq) > 0, g.integers(0, 1000, nreq), 500)
    hist[[0, 5, 127, 128, nreq - 1]] = [1000, 0, 0, 1000, 1]
    nodes[[0, 5, 127, 128, nreq - 1]] = [max_n, 0, 1, max_n, 1]
    c = make(8, hist.tolist(), nodes.tolist(), 8, 2, 64, bs, "bf16")
    whole = c["tables"].shape[1] * bs
    whole += -whole % 128
    got = call(c, split_tokens=whole)
    assert ops().get_device_error() == 0
    qs = c["q_start"].tolist()

    def alone(r):
        one = {**c, "q": c["q"][qs[r]:qs[r + 1]], "mask": c["mask"][qs[r]:qs[r + 1]], "lens": c["lens"][r:r + 1],
               "tables": c["tables"][r:r + 1],
               "q_start": torch.tensor([0, qs[r + 1] - qs[r]], dtype=torch.int32, device="cuda")}
        return call(one, split_tokens=whole)

    for r in range(nreq):
        if qs[r] < qs[r + 1]:
            assert torch.equal(got[qs[r]:qs[r + 1]], alone(r)), r
    for r in (0, 127, 128, nreq - 1):
        assert_request(c, got, r)
    bad = c["lens"].clone()
    bad[0], bad[128] = whole + 1, 2 ** 31 - 1   # past the table: refused, and first in the order
    out = torch.full_like(c["q"], 7.0)
    call({**c, "lens": bad}, out=out, split_tokens=whole)
    assert ops().get_device_error() == _lib.PA_DEVERR_CONTEXT_LEN
    skipped = torch.zeros(len(out), dtype=torch.bool, device="cuda")
    for r in (0, 128):
        skipped[qs[r]:qs[r + 1]] = True
    assert bool((out[skipped] == 7.0).all()) and torch.equal(out[~skipped], got[~skipped])


def test_empty_calls():
    c = make(7, [20], [3], 8, 2, 128, 16, "bf16")
    out = ops().verify_tree(c["q"][:0], c["q_start"][:1], c["mask"][:0], c["lens"][:0], c["kc"], c["vc"],
                            c["tables"][:0], 0.1, 4)
    assert out.shape[0] == 0 and ops().get_device_error() == 0
