"""Lengths that pass 2^31 once a partition's size is added to them: tables as wide
as the calls take, whose columns repeat a few blocks, so that a context of two
billion tokens needs no pool.

Attention over a context that repeats n0 tokens is attention over those with
every weight times how often its token comes.  The outputs' tolerance is that of
test_gpu_kv4.py (scores, their weights' rounding, the output's) and the sums: a
warp adds the weights of a partition's 16-token tiles one after another, the
merge a quarter of the partitions, each addition 2^-23 off (an MMA's sums are
cut, not rounded), in the numerator and in the denominator."""
import pytest
import torch

from test_gpu_kv4 import Batch, i32, prefill_rows

import kv4_ref as ref

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


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


def repeated(out, q, k, v, scale, n, weight_off, split):
    """out [heads, d] against the definition over k, v [n0, d] repeated to n tokens."""
    n0, d = k.shape
    times = torch.full((n0,), n // n0, dtype=torch.float64, device="cuda")
    times[:n % n0] += 1
    x = q.double() @ k.T * scale
    w = torch.exp(x - x.amax(-1, keepdim=True)) * times
    w /= w.sum(-1, keepdim=True)
    want, size = w @ v, w @ v.abs()
    score = (d + 4) * 2.0 ** -24 * abs(scale) * (q.double().abs() @ k.abs().T).amax(-1, keepdim=True)
    parts = -(-n // split)
    sums = 2 * (split // 8 + parts // 4 + 16) * 2.0 ** -23
    tol = torch.finfo(q.dtype).eps / 2 * want.abs() + (weight_off + 2.0 ** -19 + sums + 4 * score) * size + 1e-7
    assert float(want.abs().max()) > 10 * float(tol.max())  # zeros, or what was there before, would not pass
    off = (out.double() - want).abs()
    assert bool((off <= tol).all()), float((off / tol).max())


def inputs(nb, bs, heads, d):
    gen = torch.Generator(device="cuda").manual_seed(11)
    k, v = (torch.randn(nb * bs, 1, d, generator=gen, device="cuda").to(BF) for _ in range(2))
    return k, v, (torch.randn(1, heads, d, generator=gen, device="cuda") * 4).to(BF)


def test_decode_kv4_of_two_billion_tokens(ops):
    nb, bs, d, split = 64, 32, 64, 32768
    width = (2 ** 31 - 1 - 4096) // bs
    n = width * bs
    k, v, q = inputs(nb, bs, 4, d)
    kc, vc = (ops.kv4_cache(nb, bs, 1, d) for _ in range(2))
    ops.quantize_and_cache(k, v, torch.arange(nb * bs, dtype=torch.int32, device="cuda"), kc, vc)
    table = (torch.arange(width, dtype=torch.int32, device="cuda") % nb)[None].contiguous()
    for length in (n, 2 ** 31 - split, 2 ** 31 - split + 1):  # the sum below 2^31 by one, and at it
        out = torch.full_like(q, 7.0)
        ops.decode_kv4(q, kc, vc, table, i32([length]), d ** -0.5, out=out, split_tokens=split)
        assert ops.get_device_error() == 0
        held = [ref.quantized(x[:, 0])[0].cuda() for x in (k, v)]
        repeated(out[0], q[0], *held, d ** -0.5, length, 2.0 ** -11, split)


def test_decode_of_two_billion_tokens(ops):
    nb, bs, d, split = 64, 32, 64, 8192
    width = (2 ** 31 - 1) // bs
    k, v, q = inputs(nb, bs, 4, d)
    table = (torch.arange(width, dtype=torch.int32, device="cuda") % nb)[None].contiguous()
    kc, vc = k.view(nb, bs, 1, d), v.view(nb, bs, 1, d)
    for length in (width * bs, 2 ** 31 - split + 1):
        out = torch.full_like(q, 7.0)
        ops.decode(q, kc, vc, table, i32([length]), d ** -0.5, out=out, split_tokens=split)
        assert ops.get_device_error() == 0
        # weights in bf16, in the numerator and (as they are summed) in the denominator
        repeated(out[0], q[0], k[:, 0].double(), v[:, 0].double(), d ** -0.5, length, 2.0 ** -8, split)


@pytest.mark.parametrize("split", [0, 64, "two"])
def test_prefill_kv4_under_tables_of_two_billion_tokens(ops, split):
    lens, start = [6000, 300], [0, 130, 300]
    b = Batch(ops, lens, 1, 64, 32, BF)
    q = b.q(start[-1], 4)
    width = (2 ** 31 - 1 - 4096) // 32
    if split == "two":  # the second partition has no keys here
        split = (width * 32 - 1) // 64 * 64
        assert split + 6000 > 2 ** 31
    elif split == 64:   # as many partitions as scratch is had for
        width = 8192
    tables = torch.full((2, width), -1, dtype=torch.int32, device="cuda")
    tables[:, :b.tables.shape[1]] = b.tables
    out = torch.full_like(q, 7.0)
    ops.chunked_prefill_kv4(q, i32(start), b.ctx, b.kc, b.vc, tables, 0.125, 170, out=out, split_tokens=split)
    assert ops.get_device_error() == 0
    b.check(out, q, 0.125, prefill_rows(lens, start))


def test_scores_of_two_billion_tokens(ops):
    """decode_accumulate: the second pass gives a CTA a stretch of two million tokens, the last of which, and its
    rounds of 2048, end past 2^31.  A token's weight is 2^-23 off by each sum that its denominator goes through (8192 tokens, then as many partitions
    of a lane) beside its score's error."""
    nb, bs, d, split = 64, 32, 64, 8192
    width = (2 ** 31 - 1) // bs
    n = width * bs
    if torch.cuda.mem_get_info()[0] < 24 << 30:
        pytest.skip("18 GB of scores and scratch")
    k, v, q = inputs(nb, bs, 1, d)
    table = (torch.arange(width, dtype=torch.int32, device="cuda") % nb)[None].contiguous()
    scores = torch.zeros(1, 1, n, device="cuda")
    out, _ = ops.decode_accumulate(q, k.view(nb, bs, 1, d), v.view(nb, bs, 1, d), table, i32([n]), d ** -0.5, scores,
                                   split_tokens=split)
    assert ops.get_device_error() == 0
    repeated(out[0], q[0], k[:, 0].double(), v[:, 0].double(), d ** -0.5, n, 2.0 ** -8, split)
    x = (q[0].double() @ k[:, 0].double().T)[0] * d ** -0.5
    times = torch.full((nb * bs,), n // (nb * bs), dtype=torch.float64, device="cuda")
    times[:n % (nb * bs)] += 1
    w = torch.exp(x - x.max())
    w /= (w * times).sum()
    err = (d + 4) * 2.0 ** -24 * d ** -0.5 * float((q[0].double().abs() @ k[:, 0].double().abs().T).max())
    tol = 2 * (2 * 8192 + 64) * 2.0 ** -23 + 4 * err + 2.0 ** -19
    for first in (0, n // 2 // 2048 * 2048, n - 2 ** 21 - (n % 2048)):  # stretches of whole rounds of the 2048 tokens
        got = scores[0, 0, first:first + 2 ** 21].double().view(-1, nb * bs)
        assert float(((got / w - 1).abs()).max()) < tol
    last = n % (nb * bs)
    assert float((scores[0, 0, n - last:].double() / w[:last] - 1).abs().max()) < tol
    del scores
    torch.cuda.empty_cache()
