"""Norm, rotation and cache write of new tokens (pa_norm_rope_and_cache)
against a float64 form of the same, over head counts, partial and interleaved
rotations, several position axes, strided inputs, padding and bad data.

Tolerance, per element: the output is rounded once (half a step of its type,
eps/2 of the value).  Before that, in fp32: the sum of D <= 128 squares taken
in D/8 + 4 additions after a product, the factor's rsqrt (2 ulp) and halved
relative error of the sum, three products and one addition of the rotation:
under 40 roundings of 2^-24 on terms no larger than |a| + |b|, the pair's
magnitudes after the norm.  40 * 2^-24 < 2.4e-6.
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


def reference(x, w, eps, pos, table, sections, interleaved):
    """float64 rows of one of q, k, and the pair magnitudes the tolerance is relative to."""
    x = x.double().cpu()
    d, rot = x.shape[-1], table.shape[1]
    half = rot // 2
    if w is not None:
        x = x / ((x * x).mean(-1, keepdim=True) + eps).sqrt() * w.double().cpu()
    y, mag = x.clone(), x.abs()
    pos = pos.reshape(-1, x.shape[0]).long().cpu()
    axis = [a for a, n in enumerate(sections or (half,)) for _ in range(n)]
    table = table.double().cpu()
    for j in range(half):
        lo, hi = (2 * j, 2 * j + 1) if interleaved else (j, j + half)
        c, s = table[pos[axis[j]], j][:, None], table[pos[axis[j]], half + j][:, None]
        a, b = x[..., lo], x[..., hi]
        y[..., lo], y[..., hi] = a * c - b * s, b * c + a * s
        mag[..., lo] = mag[..., hi] = a.abs() + b.abs()
    return y, mag


def assert_rounded(got, want, mag, what):
    u = torch.finfo(got.dtype).eps / 2
    tol = u * want.abs() + (1 + u) * 40 * 2.0 ** -24 * mag + torch.finfo(got.dtype).smallest_normal * u
    err = (got.double().cpu() - want).abs()
    assert bool((err <= tol).all()), f"{what}: worst {float((err - tol).max())} past its tolerance"


CASES = [
    # tokens, q_heads, kv_heads, d, rot, axes/sections, norm, fused, interleaved, bs, dtype
    (1, 32, 8, 128, 128, None, True, False, False, 16, "bf16"),
    (64, 32, 8, 128, 128, None, True, True, False, 16, "bf16"),
    (77, 28, 4, 128, 64, None, False, True, False, 32, "fp16"),
    (130, 12, 12, 64, 64, (8, 12, 12), True, True, False, 8, "bf16"),
    (33, 3, 1, 64, 48, (7, 17), True, False, True, 4, "fp16"),
    (9, 64, 8, 128, 16, None, True, True, True, 16, "bf16"),
    (201, 1, 1, 128, 128, (16, 24, 24), False, False, False, 16, "fp16"),
    (2000, 5, 5, 64, 32, (0, 16, 0), True, True, False, 16, "bf16"),
]


def inputs(case, seed=0):
    t, hq, hkv, d, rot, sections, norm, fused, inter, bs, dt = case
    g = torch.Generator(device="cuda").manual_seed(seed)
    dtype = DT[dt]
    if fused:
        qkv = torch.randn(t, (hq + 2 * hkv) * d + 8, generator=g, device="cuda").to(dtype)
        q = qkv[:, :hq * d].unflatten(1, (hq, d))
        k = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
        v = qkv[:, (hq + hkv) * d:(hq + 2 * hkv) * d].unflatten(1, (hkv, d))
    else:
        q, k, v = (torch.randn(t, h, d, generator=g, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    w = [(1 + 0.2 * torch.randn(d, generator=g, device="cuda")).to(dtype) if norm else None for _ in range(2)]
    rng = np.random.default_rng(seed)
    max_pos = 5000
    axes = len(sections) if sections else 1
    pos = torch.from_numpy(rng.integers(0, max_pos, (axes, t)).astype(np.int32)).cuda()
    table = ops().rope_table(max_pos, rot, device="cuda")
    nb = t // bs + 5
    slots = rng.permutation(nb * bs)[:t].astype(np.int32)
    kc, vc = (torch.randn(nb, bs, hkv, d, generator=g, device="cuda").to(dtype) for _ in range(2))
    return q, k, v, w, pos if axes > 1 else pos[0], table, slots, kc, vc


@pytest.mark.parametrize("case", CASES, ids=[f"t{c[0]}_h{c[1]}x{c[2]}_d{c[3]}_r{c[4]}_{c[10]}" for c in CASES])
def test_matches_float64(case):
    q, k, v, w, pos, table, slots, kc, vc = inputs(case)
    sections, inter = case[5], case[8]
    if len(slots) > 3:
        slots[1] = -1  # padding: the query is still turned
    kc0, vc0 = kc.clone(), vc.clone()
    out = ops().norm_rope_and_cache(q, k, v, pos, table, torch.from_numpy(slots).cuda(), kc, vc, q_weight=w[0],
                                    k_weight=w[1], eps=1e-5, sections=sections, interleaved=inter)
    assert ops().get_device_error() == 0
    want, mag = reference(q, w[0], 1e-5, pos, table, sections, inter)
    assert_rounded(out, want, mag, "queries")
    want, mag = reference(k, w[1], 1e-5, pos, table, sections, inter)
    used = torch.from_numpy(np.nonzero(slots >= 0)[0])
    at = torch.from_numpy(slots).long()[used]
    flat = lambda c: c.view(-1, *c.shape[2:])  # noqa: E731
    assert_rounded(flat(kc).cpu()[at], want[used], mag[used], "keys")
    assert torch.equal(flat(vc).cpu()[at], v.cpu()[used])
    rest = torch.ones(flat(kc).shape[0], dtype=torch.bool)
    rest[at] = False
    assert torch.equal(flat(kc).cpu()[rest], flat(kc0).cpu()[rest])
    assert torch.equal(flat(vc).cpu()[rest], flat(vc0).cpu()[rest])


def test_in_place_queries_and_repeat():
    case = (50, 8, 2, 128, 128, None, True, False, False, 16, "bf16")
    q, k, v, w, pos, table, slots, kc, vc = inputs(case, 3)
    s = torch.from_numpy(slots).cuda()
    apart = ops().norm_rope_and_cache(q, k, v, pos, table, s, kc, vc, q_weight=w[0], k_weight=w[1])
    kc1 = kc.clone()
    same = ops().norm_rope_and_cache(q, k, v, pos, table, s, kc, vc, q_weight=w[0], k_weight=w[1], out=q)
    assert same is q and torch.equal(q, apart) and torch.equal(kc, kc1)


def test_without_norm_and_at_position_zero_it_is_the_cache_write():
    case = (70, 4, 2, 64, 64, None, False, False, False, 16, "fp16")
    q, k, v, _, pos, table, slots, kc, vc = inputs(case, 4)
    s = torch.from_numpy(slots).cuda()
    kc2, vc2 = kc.clone(), vc.clone()
    out = ops().norm_rope_and_cache(q, k, v, torch.zeros_like(pos), table, s, kc, vc)
    ops().reshape_and_cache(k, v, s, kc2, vc2)
    assert torch.equal(out, q) and torch.equal(kc, kc2) and torch.equal(vc, vc2)


def test_bad_data_is_recorded_and_skipped():
    from paged_kv_cache_76_gb300 import _lib
    case = (20, 4, 2, 64, 64, None, True, False, False, 16, "bf16")
    q, k, v, w, pos, table, slots, kc, vc = inputs(case, 5)
    good = ops().norm_rope_and_cache(q, k, v, pos, table, torch.from_numpy(slots).cuda(), kc.clone(), vc.clone())
    # a slot past the pool: only that token's K/V are skipped
    s = slots.copy()
    s[7] = kc.shape[0] * 16
    kc1, vc1 = kc.clone(), vc.clone()
    out = ops().norm_rope_and_cache(q, k, v, pos, table, torch.from_numpy(s).cuda(), kc1, vc1)
    assert ops().get_device_error() == _lib.PA_DEVERR_SLOT
    assert torch.equal(out, good)
    assert torch.equal(kc1.view(-1, 2, 64)[slots[7]], kc.view(-1, 2, 64)[slots[7]])
    # positions outside the table: that token is left alone; a padding token's are not an error
    p = pos.clone()
    p[3], p[4] = -1, table.shape[0]
    out = torch.full_like(good, 7.0)
    kc1, vc1 = kc.clone(), vc.clone()
    ops().norm_rope_and_cache(q, k, v, p, table, torch.from_numpy(slots).cuda(), kc1, vc1, out=out)
    assert ops().get_device_error() == _lib.PA_DEVERR_POSITION
    assert bool((out[3:5] == 7.0).all()) and torch.equal(out[5:], good[5:]) and torch.equal(out[:3], good[:3])
    assert torch.equal(vc1.view(-1, 2, 64)[slots[3]], vc.view(-1, 2, 64)[slots[3]])
    s = slots.copy()
    s[3] = s[4] = -1
    ops().norm_rope_and_cache(q, k, v, p, table, torch.from_numpy(s).cuda(), kc1, vc1, out=out)
    assert ops().get_device_error() == 0
    # no tokens
    empty = ops().norm_rope_and_cache(q[:0], k[:0], v[:0], pos[:0], table, torch.from_numpy(slots[:0]).cuda(), kc, vc)
    assert empty.shape == (0, 4, 64) and ops().get_device_error() == 0


def test_another_stream_capture_and_recording():
    case = (40, 8, 2, 128, 64, None, True, True, False, 16, "bf16")
    q, k, v, w, pos, table, slots, kc, vc = inputs(case, 6)
    s = torch.from_numpy(slots).cuda()
    args = (q, k, v, pos, table, s, kc, vc, w[0], w[1])
    want = ops().norm_rope_and_cache(*args)
    kc1 = kc.clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    kc.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = ops().norm_rope_and_cache(*args)
    side.synchronize()
    assert torch.equal(got, want) and torch.equal(kc.view(-1, 2, 128)[s.long()], kc1.view(-1, 2, 128)[s.long()])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = ops().norm_rope_and_cache(*args)
    got.zero_()
    graph.replay()
    assert torch.equal(got, want)
    with ops().recording() as rec:
        got = ops().norm_rope_and_cache(*args)
    got.zero_()
    rec()
    assert torch.equal(got, want)
