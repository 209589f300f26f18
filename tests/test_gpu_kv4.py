"""A cache held in 4 bits: what quantize_and_cache writes is, element by element,
the number that the definition in 64 bits gives; dequantize_kv4 gives it back
exactly; decode_kv4 is attention over those numbers.

decode_kv4 against 64 bits.  The cache's elements and q enter the products
exactly (q's elements below 2^-27 of their row's largest excepted: 2^-27 of the
score's terms, counted in the next).  A score is a sum of D products in fp32:
(D + 4) 2^-24 of sum |q k| scale off, and as much, relatively, its weight, whose
denominator carries it too (twice in all).  A weight is rounded to fp16 (2^-11
of itself), its exponential is 2^-21 off, the rest of the fp32 arithmetic (sums,
rescales, merge) 2^-20; weights that fp16 holds below its normal range are 2^-32
of the largest off each.  The output is rounded once to its type."""
import itertools

import numpy as np
import pytest
import torch

import kv4_ref as ref

pytestmark = pytest.mark.gpu
BF, HF = torch.bfloat16, torch.float16


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


def caches(ops, nb, bs, hkv, d, fill=0xFF):
    """Pools whose every byte is `fill`: 0xFF makes all they hold NaN."""
    return [torch.full_like(ops.kv4_cache(nb, bs, hkv, d), fill) for _ in range(2)]


def same(a, b):
    return bool(((a == b) | (a.isnan() & b.isnan())).all())


def check_written(ops, k, v, bs, seed=0):
    """Writes k and v to scattered slots; everything else stays."""
    T, hkv, d = k.shape
    rng = np.random.default_rng(seed)
    nb = T // bs + 3
    slots = rng.permutation(nb * bs)[:T]
    slots[rng.random(T) < 0.1] = -1
    kc, vc = caches(ops, nb, bs, hkv, d, fill=0x5A)
    ops.quantize_and_cache(k, v, i32(slots), kc, vc)
    all_slots = np.concatenate([np.arange(nb * bs), [-1]])
    back = ops.dequantize_kv4(kc, vc, i32(all_slots), d, dtype=k.dtype)
    assert ops.get_device_error() == 0
    used = np.nonzero(slots >= 0)[0]
    at = torch.from_numpy(slots[used])
    untouched = torch.full_like(kc, 0x5A).cpu()
    for cache, x, y in ((kc, k, back[0]), (vc, v, back[1])):
        held = ref.numbers(cache, bs, d).flatten(0, 1)
        want = ref.numbers(untouched, bs, d).flatten(0, 1)
        values, byte = ref.quantized(x[torch.from_numpy(used).cuda()])
        want[at] = values
        assert same(held, want)
        assert same(y[:-1].cpu().double(), want)
        assert torch.count_nonzero(y[-1]) == 0
        scales = cache.cpu()[:, :, bs * d // 2:].reshape(nb, hkv, bs, d // 16).transpose(1, 2).flatten(0, 1)
        assert torch.equal(scales[at].long(), byte)


@pytest.mark.parametrize("bs,hkv,d,dtype,T", [
    (16, 8, 128, BF, 70), (16, 4, 128, HF, 33), (4, 3, 64, BF, 19), (8, 1, 64, HF, 1), (32, 2, 128, BF, 257),
    (4, 1, 128, HF, 5), (32, 5, 64, BF, 64)])
def test_written_as_defined(ops, bs, hkv, d, dtype, T):
    gen = torch.Generator(device="cuda").manual_seed(T)
    row = torch.randn(T, 2 * hkv * d + 16, generator=gen, device="cuda")
    row *= torch.exp(3 * torch.randn(T, 1, generator=gen, device="cuda"))
    row = row.to(dtype)
    k, v = (row[:, i * hkv * d:(i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))  # views of one projection
    check_written(ops, k, v, bs)
    check_written(ops, k.contiguous(), v.contiguous(), bs, seed=1)


@pytest.mark.parametrize("T,extra,first", [(37, 8, 0), (37, 16, 8), (1, 8, 8), (21, 24, 8)])
def test_rows_that_begin_between_32_byte_lines(ops, T, extra, first):
    hkv, d = 3, 64
    row = torch.randn(T, 2 * hkv * d + extra, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").to(HF)
    k, v = (row[:, first + i * hkv * d:first + (i + 1) * hkv * d].unflatten(1, (hkv, d)) for i in range(2))
    check_written(ops, k, v, 8)
    kc, vc = caches(ops, T // 8 + 1, 8, hkv, d)
    slots = i32(np.arange(T))
    ops.quantize_and_cache(k, v, slots, kc, vc)
    want = ops.dequantize_kv4(kc, vc, slots, d, dtype=HF)
    room = torch.zeros(2, T * hkv * d + 16, dtype=HF, device="cuda")
    got = ops.dequantize_kv4(kc, vc, slots, d, dtype=HF, k=room[0, 8:8 + T * hkv * d].view(T, hkv, d),
                             v=room[1, 8:8 + T * hkv * d].view(T, hkv, d))
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    assert torch.count_nonzero(room[:, :8]) == 0 and torch.count_nonzero(room[:, 8 + T * hkv * d:]) == 0


@pytest.mark.parametrize("dtype", [BF, HF])
def test_ties_ends_and_values_that_are_not_finite(ops, dtype):
    d = 64
    rows = []
    for s in (2.0 ** -17, 2.0 ** -15, 2.0 ** -14, 0.0078125, 1.0, 1.125, 1.875, 3.25, 1000.0, 10240.0):
        # every midpoint of two levels and a hair to each side of it, beside the largest, 6 s
        mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0], dtype=torch.float64) * s
        t = mids.to(dtype)
        up, down = (torch.nextafter(t, torch.full_like(t, w)) for w in (float("inf"), 0.0))
        rows.append(torch.cat([t, -t, up.clamp(max=float(t[-1])), t, down, -down, t, t.flip(0)]))
    for top in (0.0, 2.0 ** -24, 6 * 2.0 ** -18, 9 * 2.0 ** -18, 6 * 2.0 ** -18 * 1.0078125, 61440.0, 65504.0,
                float("inf"), -float("inf"), float("nan")):
        x = torch.linspace(-1, 1, d, dtype=torch.float64) * min(abs(top), 1.0) if np.isfinite(top) else torch.ones(d)
        x[17] = top
        rows.append(x.to(dtype))
    if dtype == BF:
        x = torch.full((d,), 3.0e38).to(dtype)
        x[5], x[40] = -1.0e-38, 1.0
        rows.append(x)
    # scales at their own midpoints: 6 (1 + (2i+1)/16) 2^e, where the type holds it
    for e, i in itertools.product((-16, -14, -3, 0, 4), range(8)):
        x = torch.randn(d, generator=torch.Generator().manual_seed(i)) * 2.0 ** e
        x = x.clamp(-2.0 ** e, 2.0 ** e)
        x[::16] = 6 * (1 + (2 * i + 1) / 16) * 2.0 ** e
        rows.append(x.to(dtype))
    x = torch.stack([r.to(dtype) for r in rows]).cuda().view(-1, 1, d)
    check_written(ops, x, x.flip(0).contiguous(), 16)


def test_slots_past_the_pool(ops):
    k = torch.randn(4, 2, 64, device="cuda").to(BF)
    kc, vc = caches(ops, 3, 8, 2, 64)
    ops.quantize_and_cache(k, k, i32([0, 24, 5, 2 ** 30]), kc, vc)
    assert ops.get_device_error() == 3
    got, _ = ops.dequantize_kv4(kc, vc, i32([0, 5, 1]), 64)
    want, _ = ref.quantized(k[[0, 2]])
    assert same(got[:2].cpu().double(), want) and bool(got[2].isnan().all())
    assert ops.get_device_error() == 0
    got, _ = ops.dequantize_kv4(kc, vc, i32([24, 5]), 64)
    assert ops.get_device_error() == 3
    assert torch.count_nonzero(got[0]) == 0 and same(got[1].cpu().double(), want[1])
    ops.quantize_and_cache(k[:0], k[:0], i32(np.zeros(0)), kc, vc)  # nothing to write


class Batch:
    """Sequences of given lengths over a scattered pool that holds NaN everywhere else."""

    def __init__(self, ops, lens, hkv, d, bs, dtype, seed=0, spread=1.0):
        self.lens, self.bs, self.d, self.dtype = lens, bs, d, dtype
        rng = np.random.default_rng(seed)
        self.gen = torch.Generator(device="cuda").manual_seed(seed)
        blocks = [-(-n // bs) for n in lens]
        nb = sum(blocks) + 3
        perm = rng.permutation(nb)
        self.kc, self.vc = caches(ops, nb, bs, hkv, d)
        width = max(max(blocks), 1) + 1
        tables = np.full((len(lens), width), -7)
        at = 0
        for r, n in enumerate(blocks):
            tables[r, :n] = perm[at:at + n]
            at += n
        self.tables, self.ctx = i32(tables), i32(lens)
        self.k, self.v = [], []
        for r, n in enumerate(lens):
            t = np.arange(n)
            x = [(torch.randn(n, hkv, d, generator=self.gen, device="cuda") * spread).to(dtype) for _ in range(2)]
            ops.quantize_and_cache(x[0], x[1], i32(tables[r, t // bs] * bs + t % bs), self.kc, self.vc)
            self.k.append(ref.quantized(x[0])[0].cuda())
            self.v.append(ref.quantized(x[1])[0].cuda())

    def q(self, *shape, size=2.0):
        return (torch.randn(*shape, self.d, generator=self.gen, device="cuda") * size).to(self.dtype)

    def check(self, out, q, scale, rows_of):
        """rows_of(r): (rows of q and out of request r as a slice, tokens each of them sees)."""
        hq = q.shape[-2]
        q, out = q.reshape(-1, hq, self.d), out.reshape(-1, hq, self.d)
        u = torch.finfo(self.dtype).eps / 2
        for r, n in enumerate(self.lens):
            at, seen = rows_of(r)
            mask = torch.arange(max(n, 1), device="cuda")[None] < torch.tensor(seen, device="cuda")[:, None]
            for h in range(hq):
                hk = h // (hq // self.k[r].shape[1])
                k, v = (x[r][:, hk] if n else torch.zeros(1, self.d, dtype=torch.float64, device="cuda")
                        for x in (self.k, self.v))
                x = q[at, h].double()
                want, size = ref.attend(x, k, v, scale, mask)
                err = (self.d + 4) * 2.0 ** -24 * abs(scale) * (x.abs() @ k.abs().T).amax(-1, keepdim=True)
                tol = u * want.abs() + (2.0 ** -11 + 2.0 ** -19 + 4 * err) * size + n * 2.0 ** -32 * v.abs().max() + 1e-7
                off = (out[at, h].double() - want).abs()
                assert bool((off <= tol).all()), (r, h, float((off / tol).max()))


def decode_rows(lens, ql):
    def rows_of(r):
        return slice(r * ql, (r + 1) * ql), [max(lens[r] - (ql - 1 - i), 0) for i in range(ql)]
    return rows_of


LENS = [0, 1, 2, 15, 16, 17, 31, 32, 33, 100, 257, 700]


@pytest.mark.parametrize("hq,hkv,d,bs,dtype", [
    (32, 8, 128, 16, BF), (28, 4, 128, 16, HF), (8, 1, 64, 4, BF), (12, 12, 64, 8, HF), (16, 1, 128, 32, BF),
    (18, 2, 64, 32, BF), (8, 2, 128, 4, HF), (4, 2, 128, 8, BF)])
@pytest.mark.parametrize("split", [0, 32, 256])
def test_decode(ops, hq, hkv, d, bs, dtype, split):
    b = Batch(ops, LENS, hkv, d, bs, dtype)
    q = b.q(len(LENS), hq)
    scale = d ** -0.5
    out = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, scale, split_tokens=split)
    assert ops.get_device_error() == 0
    b.check(out, q, scale, decode_rows(LENS, 1))
    again = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, scale, split_tokens=split)
    assert torch.equal(out, again)


@pytest.mark.parametrize("hq,hkv,d,bs,dtype,ql", [
    (32, 8, 128, 16, BF, 4), (28, 4, 128, 16, HF, 2), (8, 8, 64, 4, BF, 32), (8, 1, 64, 8, HF, 3),
    (16, 1, 128, 32, BF, 2), (12, 4, 128, 16, BF, 7), (4, 4, 128, 8, BF, 1)])
@pytest.mark.parametrize("split", [0, 32])
def test_several_queries(ops, hq, hkv, d, bs, dtype, ql, split):
    b = Batch(ops, LENS, hkv, d, bs, dtype)
    q = b.q(len(LENS), ql, hq)
    scale = d ** -0.5
    out = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, scale, split_tokens=split)
    assert ops.get_device_error() == 0
    b.check(out, q, scale, decode_rows(LENS, ql))


@pytest.mark.parametrize("size,spread", [(1e-30, 1.0), (3e4, 1.0), (2.0, 3e-3), (40.0, 5.0), (0.0, 1.0)])
def test_queries_and_caches_of_any_size(ops, size, spread):
    b = Batch(ops, [700, 33, 90], 2, 128, 16, BF, spread=spread)
    q = b.q(3, 8, size=size)
    scale = 0.09 if size < 100 else 1e-5
    out = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, scale, split_tokens=64)
    b.check(out, q, scale, decode_rows(b.lens, 1))
    out = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, -scale)
    b.check(out, q, -scale, decode_rows(b.lens, 1))


@pytest.mark.parametrize("split", [0, 32])
def test_a_token_that_is_not_a_number(ops, split):
    """It reaches the queries that see it and no other, in V only the elements of its group."""
    lens, ql, hq, hkv, d = [64, 40, 35], 6, 8, 2, 128
    b = Batch(ops, lens, hkv, d, 16, BF)
    q = b.q(3, ql, hq)
    clean = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, split_tokens=split)
    # request 0: V of its token 61 (query 2 + ...) ; request 1: K of token 39; request 2: V of token 3
    bad = torch.ones(1, hkv, d, device="cuda").to(BF)
    badv, badk = bad.clone(), bad.clone()
    badv[0, 1, 37] = float("inf")

    def slot(r, t):
        return int(b.tables[r, t // 16]) * 16 + t % 16
    kc, vc = b.kc.clone(), b.vc.clone()
    keep = ops.dequantize_kv4(b.kc, b.vc, i32([slot(0, 61), slot(2, 3)]), d)
    badk[0, 0, 5] = float("nan")
    ops.quantize_and_cache(keep[0][0:1].contiguous(), badv, i32([slot(0, 61)]), kc, vc)
    ops.quantize_and_cache(keep[0][1:2].contiguous(), badv, i32([slot(2, 3)]), kc, vc)
    keep = ops.dequantize_kv4(b.kc, b.vc, i32([slot(1, 39)]), d)
    ops.quantize_and_cache(badk, keep[1], i32([slot(1, 39)]), kc, vc)
    out = ops.decode_kv4(q, kc, vc, b.tables, b.ctx, 0.1, split_tokens=split)
    for i in range(ql):
        sees = 64 - (ql - 1 - i) > 61
        nan = out[0, i].isnan()
        assert bool(nan[4:, 32:48].all()) == sees
        nan[4:, 32:48] = False
        assert not bool(nan.any())
        if not sees:
            assert torch.equal(out[0, i], clean[0, i])
        sees = i == ql - 1
        assert bool(out[1, i, :4].isnan().all()) == sees and not bool(out[1, i, 4:].isnan().any())
        assert sees or torch.equal(out[1, i], clean[1, i])
        assert bool(out[2, i, 4:, 32:48].isnan().all()) and not bool(out[2, i, :4].isnan().any())


def test_bad_blocks_and_lengths(ops):
    b = Batch(ops, [40, 90, 16], 2, 128, 16, BF)
    q = b.q(3, 8)
    good = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1)
    assert ops.get_device_error() == 0
    t = b.tables.clone()
    t[1, 2] = 10 ** 6
    out = ops.decode_kv4(q, b.kc, b.vc, t, b.ctx, 0.1)
    assert ops.get_device_error() == 1
    assert torch.equal(out[0], good[0]) and torch.equal(out[2], good[2])
    want, _ = ref.attend(q[1, :4].double(), torch.cat([b.k[1][:32, 0], 0 * b.k[1][:16, 0], b.k[1][48:, 0]]),
                         torch.cat([b.v[1][:32, 0], 0 * b.v[1][:16, 0], b.v[1][48:, 0]]), 0.1,
                         torch.ones(4, 90, dtype=torch.bool, device="cuda"))
    assert float((out[1, :4].double() - want).abs().max()) < 0.02
    for bad in (-1, 16 * t.shape[1] + 1):
        n = b.ctx.clone()
        n[0] = bad
        out = ops.decode_kv4(q, b.kc, b.vc, b.tables, n, 0.1)
        assert ops.get_device_error() in (1, 2)
        assert torch.equal(out[1:], good[1:])


def prefill_rows(lens, start):
    def rows_of(r):
        n = start[r + 1] - start[r]
        return slice(start[r], start[r + 1]), [lens[r] - n + i + 1 for i in range(n)]
    return rows_of


CHUNKS = [(1, 1), (130, 7), (64, 64), (200, 33), (700, 0), (65, 65), (0, 0), (257, 1), (300, 129)]  # (context, chunk)


@pytest.mark.parametrize("hq,hkv,d,bs,dtype", [
    (32, 8, 128, 16, BF), (28, 4, 128, 16, HF), (8, 1, 64, 4, BF), (12, 12, 64, 8, HF), (16, 1, 128, 32, BF),
    (18, 2, 64, 32, BF), (8, 2, 128, 4, HF), (4, 2, 128, 8, BF)])
@pytest.mark.parametrize("split", [0, 64, 256])
def test_prefill(ops, hq, hkv, d, bs, dtype, split):
    lens = [n for n, _ in CHUNKS]
    start = np.concatenate([[0], np.cumsum([c for _, c in CHUNKS])])
    b = Batch(ops, lens, hkv, d, bs, dtype)
    q = b.q(int(start[-1]) + 2, hq)
    scale = d ** -0.5
    out = torch.full_like(q, 7.0)
    ops.chunked_prefill_kv4(q, i32(start), b.ctx, b.kc, b.vc, b.tables, scale, 140, out=out, split_tokens=split)
    assert ops.get_device_error() == 0
    assert bool((out[-2:] == 7).all())  # rows behind the last chunk
    b.check(out, q, scale, prefill_rows(lens, start))
    again = ops.chunked_prefill_kv4(q, i32(start), b.ctx, b.kc, b.vc, b.tables, scale, 140, split_tokens=split)
    assert torch.equal(out[:-2], again[:-2])


@pytest.mark.parametrize("size,spread,scale", [(1e-30, 1.0, 0.09), (1e-30, 1.0, 1e-12), (3e4, 1.0, 1e-5), (2.0, 3e-3, 0.09),
                                               (40.0, 5.0, 0.09), (2.0, 1.0, -0.09)])
def test_prefill_of_any_size(ops, size, spread, scale):
    b = Batch(ops, [400, 70], 2, 128, 16, BF, spread=spread)
    q = b.q(100 + 70, 8, size=size)
    for split in (0, 64):
        out = ops.chunked_prefill_kv4(q, i32([0, 100, 170]), b.ctx, b.kc, b.vc, b.tables, scale, 100, split_tokens=split)
        b.check(out, q, scale, prefill_rows([400, 70], [0, 100, 170]))
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("split", [0, 64])
def test_prefill_past_a_token_that_is_not_a_number(ops, split):
    lens, hq, hkv, d, n = [150, 300], 8, 2, 128, 150
    b = Batch(ops, lens, hkv, d, 16, BF)
    start = [0, n, n + 100]
    q = b.q(start[-1], hq)
    args = (q, i32(start), b.ctx)
    clean = ops.chunked_prefill_kv4(*args, b.kc, b.vc, b.tables, 0.1, n, split_tokens=split)

    def slot(r, t):
        return i32([int(b.tables[r, t // 16]) * 16 + t % 16])
    keep = [ops.dequantize_kv4(b.kc, b.vc, slot(r, t), d) for r, t in ((0, 77), (1, 250))]
    badv, badk = keep[0][1].clone(), keep[1][0].clone()  # but for one element what the cache holds: written as it is
    badv[0, 1, 37], badk[0, 0, 5] = float("inf"), float("nan")
    kc, vc = b.kc.clone(), b.vc.clone()
    ops.quantize_and_cache(keep[0][0], badv, slot(0, 77), kc, vc)   # seen by queries 77 on
    ops.quantize_and_cache(badk, keep[1][1], slot(1, 250), kc, vc)  # by queries 50 on of the second chunk
    out = ops.chunked_prefill_kv4(*args, kc, vc, b.tables, 0.1, n, split_tokens=split)
    nan = out.isnan()
    assert bool(nan[77:n, 4:, 32:48].all()) and bool(nan[n + 50:, :4].all())
    nan[77:n, 4:, 32:48] = False
    nan[n + 50:, :4] = False
    assert not bool(nan.any())
    for got, want in ((out[:77], clean[:77]), (out[77:n, :4], clean[77:n, :4]), (out[n:n + 50], clean[n:n + 50]),
                      (out[n + 50:, 4:], clean[n + 50:, 4:])):
        assert torch.equal(got, want)


def test_prefill_refuses_requests(ops):
    b = Batch(ops, [60, 90, 40], 2, 128, 16, BF)
    start = [0, 10, 30, 45]
    q = b.q(45, 8)
    good = ops.chunked_prefill_kv4(q, i32(start), b.ctx, b.kc, b.vc, b.tables, 0.1, 20)
    assert ops.get_device_error() == 0
    for lens, starts, most in [([60, 19, 40], start, 20), ([60, 10 ** 6, 40], start, 20), ([60, 90, 40], start, 17),
                               ([60, 90, 40], [0, 10, 4, 45], 20), ([60, 90, 40], [0, 10, 60, 45], 20)]:
        out = torch.full_like(q, 7.0)
        ops.chunked_prefill_kv4(q, i32(starts), i32(lens), b.kc, b.vc, b.tables, 0.1, most, out=out)
        assert ops.get_device_error() == 5
        assert torch.equal(out[:10], good[:10])
        assert bool((out[10:30] == 7).all()) or starts != start
    t = b.tables.clone()
    t[1, 1] = -3
    out = ops.chunked_prefill_kv4(q, i32(start), b.ctx, b.kc, b.vc, t, 0.1, 20)
    assert ops.get_device_error() == 1
    assert torch.equal(out[:10], good[:10]) and torch.equal(out[30:], good[30:])


@pytest.mark.parametrize("split", [0, 64])
def test_prefill_refuses_the_most_negative_length(ops, split):
    b = Batch(ops, [60, 90], 2, 128, 16, BF)
    q = b.q(30, 8)
    good = ops.chunked_prefill_kv4(q, i32([0, 10, 30]), b.ctx, b.kc, b.vc, b.tables, 0.1, 20, split_tokens=split)
    for length in (-2 ** 31, -2 ** 31 + 19, -1):  # the first two less 20 do not fit 32 bits
        out = torch.full_like(q, 7.0)
        ops.chunked_prefill_kv4(q, i32([0, 10, 30]), i32([60, length]), b.kc, b.vc, b.tables, 0.1, 20, out=out,
                                split_tokens=split)
        assert ops.get_device_error() == 5
        assert torch.equal(out[:10], good[:10]) and bool((out[10:] == 7).all())


def test_another_stream_a_capture_and_a_recording(ops):
    b = Batch(ops, [300, 5, 77], 2, 128, 16, BF)
    q = b.q(3, 8)
    want = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    out, k = torch.zeros_like(want), b.q(1, 2)
    kc, vc = b.kc.clone(), b.vc.clone()
    g = torch.cuda.CUDAGraph()
    slot = i32([int(b.tables[1, 0]) * 16 + 4])
    with torch.cuda.graph(g):
        ops.quantize_and_cache(k, k, slot, kc, vc)
        ops.decode_kv4(q, kc, vc, b.tables, b.ctx, 0.1, out=out)
    with ops.recording() as rec:
        again = ops.decode_kv4(q, kc, vc, b.tables, b.ctx, 0.1)
    for seed in range(2):
        k.copy_(b.q(1, 2))
        g.replay()
        rec()
        ops.quantize_and_cache(k, k, slot, b.kc, b.vc)
        want = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1)
        assert torch.equal(out, want) and torch.equal(again, want)
    assert ops.get_device_error() == 0


def test_two_calls_at_once_and_a_given_workspace(ops):
    b = Batch(ops, [700, 5, 300], 2, 128, 16, BF)
    q, qp = b.q(3, 8), b.q(60, 8)
    start = i32([0, 30, 35, 60])
    # split_tokens 32: partials and a merge; 64: twelve partitions, a cluster
    want = {n: ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, split_tokens=n) for n in (32, 64)}
    wantp = ops.chunked_prefill_kv4(qp, start, b.ctx, b.kc, b.vc, b.tables, 0.1, 30, split_tokens=64)
    torch.cuda.synchronize()
    streams, got = [torch.cuda.Stream() for _ in range(4)], []
    for _ in range(6):
        for i, s in enumerate(streams):
            with torch.cuda.stream(s):
                if i % 2:
                    n = 32 if i == 1 else 64
                    got.append((ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, split_tokens=n), want[n]))
                else:
                    got.append((ops.chunked_prefill_kv4(qp, start, b.ctx, b.kc, b.vc, b.tables, 0.1, 30,
                                                        split_tokens=64), wantp))
    torch.cuda.synchronize()
    assert all(torch.equal(g, w) for g, w in got)
    ws = torch.empty(1 << 24, dtype=torch.uint8, device="cuda")
    for _ in range(3):  # one scratch for calls in order
        assert torch.equal(ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, split_tokens=32, workspace=ws), want[32])
        assert torch.equal(ops.chunked_prefill_kv4(qp, start, b.ctx, b.kc, b.vc, b.tables, 0.1, 30, split_tokens=64,
                                                   workspace=ws), wantp)
    from paged_kv_cache_76_gb300 import PAError
    with pytest.raises(PAError):
        ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, split_tokens=32, workspace=ws[:256])
    assert ops.get_device_error() == 0


@pytest.mark.parametrize("hq,hkv,d,bs,ql", [(8, 1, 128, 16, 1), (4, 1, 64, 4, 1), (16, 1, 128, 32, 2), (8, 2, 128, 8, 3)])
@pytest.mark.parametrize("parts", [2, 5, 13, 16, 17])
def test_partitions_that_join(ops, hq, hkv, d, bs, ql, parts):
    """Clusters of every size beside the next that takes a merge; contexts that end in any of the partitions."""
    most = 64 * parts - bs  # tables have a column more
    lens = [most, 0, 1, 64, 65, 64 * (parts // 2) + 3]
    b = Batch(ops, lens, hkv, d, bs, BF)
    q = b.q(len(lens), ql, hq)
    size = ops.decode_kv4_workspace_size(len(lens), ql, hq, hkv, d, b.tables.shape[1], bs, 64)
    assert (size == 0) == (parts <= 16)
    out = ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, split_tokens=64)
    assert ops.get_device_error() == 0
    b.check(out, q, 0.1, decode_rows(lens, ql))
    assert torch.equal(out, ops.decode_kv4(q, b.kc, b.vc, b.tables, b.ctx, 0.1, split_tokens=64))


def test_wide_tables_and_many_requests(ops):
    """Tables wider than the contexts, and as many requests as a call takes in one dimension of its grid."""
    b = Batch(ops, [33, 0, 61], 1, 64, 16, BF)
    q = b.q(3, 4)
    wide = torch.full((3, 5000), -1, dtype=torch.int32, device="cuda")
    wide[:, :b.tables.shape[1]] = b.tables
    out = ops.decode_kv4(q, b.kc, b.vc, wide, b.ctx, 0.1)
    b.check(out, q, 0.1, decode_rows(b.lens, 1))
    n = 65535
    big = b.tables[[0, 2]].repeat(n // 2 + 1, 1)[:n].contiguous()
    lens = b.ctx[[0, 2]].repeat(n // 2 + 1)[:n].contiguous()
    qs = q[[0, 2]].repeat(n // 2 + 1, 1, 1)[:n].contiguous()
    got = ops.decode_kv4(qs, b.kc, b.vc, big, lens, 0.1)
    for i in range(2):
        mine = got[i::2]
        assert torch.equal(mine, mine[:1].expand_as(mine))
        assert float((mine[0].float() - out[2 * i].float()).abs().max()) < 0.01
    start = torch.arange(n + 1, dtype=torch.int32, device="cuda")
    pre = ops.chunked_prefill_kv4(qs, start, lens, b.kc, b.vc, big, 0.1, 1)
    for i in range(2):
        mine = pre[i::2]
        assert torch.equal(mine, mine[:1].expand_as(mine))
        assert float((mine[0].float() - out[2 * i].float()).abs().max()) < 0.01
    assert ops.get_device_error() == 0


def test_a_cache_past_two_gigabytes(ops):
    """Pages whose byte offset passes 32 bits."""
    hkv, d, bs = 8, 128, 16
    nb = 2 ** 32 // (hkv * bs * 72) + 40
    kc, vc = (torch.empty(nb, hkv, bs * 72, dtype=torch.uint8, device="cuda") for _ in range(2))
    ids = [nb - 1, 3, nb - 17, nb // 2 + 1]
    n = 61
    gen = torch.Generator(device="cuda").manual_seed(3)
    k, v = (torch.randn(n, hkv, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    t = np.arange(n)
    slots = i32(np.asarray(ids)[t // bs] * bs + t % bs)
    ops.quantize_and_cache(k, v, slots, kc, vc)
    back = ops.dequantize_kv4(kc, vc, slots, d)
    assert same(back[0].cpu().double(), ref.quantized(k)[0]) and same(back[1].cpu().double(), ref.quantized(v)[0])
    q = (torch.randn(1, 32, d, generator=gen, device="cuda") * 2).to(BF)
    out = ops.decode_kv4(q, kc, vc, i32([ids]), i32([n]), 0.1)
    small = [c[torch.tensor(ids, device="cuda")].contiguous() for c in (kc, vc)]
    assert torch.equal(out, ops.decode_kv4(q, *small, i32([[0, 1, 2, 3]]), i32([n]), 0.1))
    assert ops.get_device_error() == 0
