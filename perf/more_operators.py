"""Cases of a paged cache held in 4 bits, and of pages forked on the device.

Four operators of the library, each in its plain form (elementary torch
operations in 32 bits, rounded once at the end) and as the library's call:

* ``write``: new keys and values into a cache of 4-bit elements with a scale
  for every 16 (``ops.quantize_and_cache``), and the cache read back in 16
  bits (``ops.dequantize_kv4``);
* ``decode``: attention of one query a request, or of a few causal ones, over
  that cache (``ops.decode_kv4``);
* ``prefill``: attention of prompt chunks over it (``ops.chunked_prefill_kv4``);
* ``fork``: sequences continued from others (a beam search's step, several
  samples of a prompt): Block Tables that share full pages, pages to copy and
  pages for the next tokens (``ops.fork_blocks``), and the copies in the caches
  of several layers (``ops.copy_pages``).

Sizes follow the workloads of this repository (32/8, 64/8 and 28/4 heads of
128, 16-token blocks, contexts of hundreds to 131072 tokens) and odd ones
around them.

An element is one of 0, 0.5, 1, 1.5, 2, 3, 4, 6 with a sign (nearest, ties to
the even code), times the scale of its 16 neighbours along the head: the
largest magnitude / 6, rounded to three bits behind the leading one (a scale's
byte is bits 14..7 of the same number in fp16; at most 10240; 2^-17 apart below
2^-14).  A page is one block of one head: ``[block_size][head_dim / 2]`` bytes
of codes, the even element in the low half, then ``[block_size][head_dim / 16]``
scales; a cache is ``[num_blocks, kv_heads, page bytes]``.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GOLDEN = 0.6180339887498949
LEVELS = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
TOP_SCALE = 226  # 10240


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step's new tokens of a batch
        dict(name="write_decode_64", op="write", tokens=64, hq=32, hkv=8, d=128, bs=16, fused=True, dtype="bf16"),
        # one prefill step, k and v as views of a fused projection's rows
        dict(name="write_prefill_8192", op="write", tokens=8192, hq=32, hkv=8, d=128, bs=16, fused=True, dtype="bf16"),
        # few requests, odd contexts: latency
        dict(name="decode_small", op="decode", batch=4, lo=301, hi=1501, q_len=1, hq=28, hkv=4, d=128, bs=16,
             dtype="bf16"),
        # a serving batch
        dict(name="decode_64", op="decode", batch=64, lo=509, hi=4079, q_len=1, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # the same batch verifying three drafted tokens a request
        dict(name="verify_64", op="decode", batch=64, lo=509, hi=4079, q_len=4, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # long contexts: the keys have to be split over the GPU
        dict(name="decode_long", op="decode", batch=8, lo=32768, hi=131009, q_len=1, hq=64, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # short chunks of a few prompts beside others' decode steps
        dict(name="prefill_short", op="prefill", reqs=4, clo=37, chi=131, lo=301, hi=1501, hq=28, hkv=4, d=128, bs=16,
             dtype="bf16"),
        # one step of chunked prefill: eight chunks of different lengths
        dict(name="prefill_chunks", op="prefill", reqs=8, clo=257, chi=768, lo=509, hi=4079, hq=32, hkv=8, d=128,
             bs=16, dtype="bf16"),
        # the last chunk of a long prompt
        dict(name="prefill_long", op="prefill", reqs=1, clo=2048, chi=2048, lo=32768, hi=32768, hq=64, hkv=8, d=128,
             bs=16, dtype="bf16"),
        # four requests of four beams
        dict(name="fork_16", op="fork", reqs=4, beams=4, lo=301, hi=1501, hkv=4, d=128, bs=16, layers=2, dtype="bf16"),
        # a beam search's step of 64 requests, the copies in two layers
        dict(name="fork_512", op="fork", reqs=64, beams=8, lo=509, hi=4079, hkv=8, d=128, bs=16, layers=2,
             dtype="bf16"),
        # beams over long contexts: tables of thousands of blocks
        dict(name="fork_long", op="fork", reqs=8, beams=8, lo=32768, hi=131009, hkv=1, d=64, bs=16, layers=2,
             dtype="bf16"),
    ]


def draw(rng):
    op = rng.choice(["write", "decode", "decode", "prefill", "fork"])
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    d = rng.choice([128, 128, 64])
    hq, hkv = rng.choice([(32, 8), (28, 4), (64, 8), (16, 2), (8, 1), (12, 12)])
    bs = rng.choice([4, 8, 16, 16, 32])
    if op == "write":
        return dict(op=op, tokens=log(1, 8192), hq=hq, hkv=min(hkv, 8), d=d, bs=bs, fused=rng.random() < 0.5,
                    dtype=dtype)
    if op == "decode":
        batch = log(1, 64)
        hi = log(40, min(131072, 400000 // batch))
        most = max(1, 32 // (hq // hkv))
        return dict(op=op, batch=batch, lo=max(1, hi // rng.choice([2, 8, 50])), hi=hi,
                    q_len=1 if rng.random() < 0.6 else log(1, most), hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype)
    if op == "prefill":
        reqs = log(1, 16)
        chi = log(2, min(2048, 4096 // reqs))
        hi = log(20, min(65536, int(3e9 / (hq * reqs * chi))))
        return dict(op=op, reqs=reqs, clo=max(1, chi // rng.choice([1, 2, 8])), chi=chi, lo=hi // rng.choice([2, 8, 50]),
                    hi=hi, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype)
    reqs, beams = log(1, 64), rng.choice([1, 2, 3, 4, 8])
    hi = log(20, min(131072, 200000 // reqs))
    return dict(op=op, reqs=reqs, beams=beams, lo=max(1, hi // rng.choice([2, 8, 50])), hi=hi, hkv=rng.choice([1, 4]),
                d=d, bs=bs, layers=rng.choice([1, 2, 3]), dtype=dtype)


def _spread(n, lo, hi, phase):
    """n whole numbers over [lo, hi], the same for every seed (a low-discrepancy sequence)."""
    return (lo + np.floor((hi - lo + 1) * ((np.arange(n) * GOLDEN + phase) % 1.0))).astype(np.int64)


def _lens(case):
    """(context lengths, queries) of the requests; a chunk is counted in its context."""
    if case["op"] == "prefill":
        chunk = _spread(case["reqs"], case["clo"], case["chi"], 0.25)
        return _spread(case["reqs"], case["lo"], case["hi"], 0.5) + chunk, chunk
    if case["op"] == "fork":
        lens = _spread(case["reqs"], case["lo"], case["hi"], 0.5)
        return lens, np.ones_like(lens)
    lens = _spread(case["batch"], case["lo"], case["hi"], 0.5)
    return lens, np.full_like(lens, case["q_len"])


def work(case):
    op, hkv, d = case["op"], case["hkv"], case["d"]
    head = d // 2 + d // 16  # bytes of a token of one head
    if op == "write":
        t = case["tokens"]
        slots = _write_blocks(case) * case["bs"]
        # k and v read, written as pages; the pages read, given out in 16 bits
        return {"bytes": 2 * t * hkv * (2 * d + head) + 2 * slots * hkv * (head + 2 * d) + 4 * t,
                "flops": 4 * t * hkv * d + 2 * slots * hkv * d}
    lens, rows = _lens(case)
    if op == "fork":
        width, n = int((-(-lens // case["bs"])).sum()) * case["beams"], case["reqs"] * case["beams"]
        page = 2 * case["bs"] * hkv * d
        copies = case["reqs"] * (case["beams"] - 1) // 2  # about as many beams as this continue from another's page
        return {"bytes": 8 * width + 28 * n + 4 * case["layers"] * copies * page, "flops": 0}
    hq, total = case["hq"], int(lens.sum())
    seen = int((rows * lens - rows * (rows - 1) // 2).sum())
    return {"bytes": 2 * total * hkv * head + 4 * int(rows.sum()) * hq * d + 4 * total // case["bs"],
            "flops": 4 * seen * hq * d}


# --------------------------------------------------------------------------
# the 4-bit cache in torch
# --------------------------------------------------------------------------
def _scale_bytes(top):
    """Byte of the scale of groups whose largest magnitude is `top` (fp32)."""
    f = top / 6.0
    u = f.view(torch.int32)
    normal = ((u + 0x7FFFF + ((u >> 20) & 1)) >> 20) - (112 << 3)
    small = torch.round(f * 2.0 ** 17).to(torch.int32)
    return torch.where(f < 2.0 ** -14, small, normal).clamp_max(TOP_SCALE)


def _scale_values(byte):
    return (byte.to(torch.int16) << 7).view(torch.float16).float()


def _encode(x):
    """x fp32 [..., d]: codes [..., d] (0..15) and scale bytes [..., d / 16]."""
    g = x.unflatten(-1, (-1, 16))
    byte = _scale_bytes(g.abs().amax(-1))
    s = _scale_values(byte)[..., None]
    y = torch.where(s > 0, g / torch.where(s > 0, s, torch.ones_like(s)), torch.zeros_like(g))
    m = y.abs()
    code = (m > 0.25).to(torch.uint8)
    for bound, even in ((0.75, True), (1.25, False), (1.75, True), (2.5, False), (3.5, True), (5.0, False)):
        code += (m >= bound) if even else (m > bound)
    return (code + 8 * (y < 0).to(torch.uint8)).flatten(-2), byte.to(torch.uint8)


def _values(code, byte):
    """The numbers that codes [..., d] and scale bytes [..., d / 16] stand for, in 32 bits."""
    level = torch.tensor(LEVELS + [-x for x in LEVELS], device=code.device)
    v = torch.index_select(level, 0, code.flatten().to(torch.int32)).view(code.shape)
    return (v.unflatten(-1, (-1, 16)) * _scale_values(byte)[..., None]).flatten(-2)


def _pack(code, byte):
    """codes [n, bs, heads, d] and scales [n, bs, heads, d / 16] as pages [n, heads, bytes]."""
    code, byte = code.transpose(1, 2), byte.transpose(1, 2)
    both = code[..., 0::2] | code[..., 1::2] << 4
    return torch.cat([both.flatten(2), byte.flatten(2)], -1).contiguous()


def _unpack(pages, bs, d):
    """Pages [n, heads, bytes] as codes [n, bs, heads, d] and scales [n, bs, heads, d / 16]."""
    cut = bs * d // 2
    both = pages[..., :cut].unflatten(-1, (bs, d // 2)).transpose(1, 2)
    code = torch.stack([both & 15, both >> 4], -1).flatten(-2)
    return code, pages[..., cut:].unflatten(-1, (bs, d // 16)).transpose(1, 2)


def _cache(gen, blocks, case):
    """A cache of normal values, made a few blocks at a time."""
    hkv, d, bs = case["hkv"], case["d"], case["bs"]
    out = torch.empty((blocks, hkv, bs * d * 9 // 16), dtype=torch.uint8, device="cuda")
    step = max(1, (1 << 25) // (bs * hkv * d))
    for b in range(0, blocks, step):
        n = min(step, blocks - b)
        x = torch.randn((n, bs, hkv, d), generator=gen, device="cuda")
        out[b:b + n] = _pack(*_encode(x))
    return out


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _i32(a):
    return torch.from_numpy(np.ascontiguousarray(a).astype(np.int32)).cuda()


def _tables(rng, lens, bs):
    """Block Tables of sequences scattered over a pool a tenth larger than they need."""
    blocks = -(-lens // bs)
    pool = int(blocks.sum() * 1.1) + 4
    perm = rng.permutation(pool)
    starts = np.cumsum(blocks) - blocks
    cols = np.arange(int(blocks.max()))[None]
    at = np.minimum(starts[:, None] + cols, pool - 1)
    return np.where(cols < blocks[:, None], perm[at], -1), pool


def _normal(gen, shape, dtype, scale=1.0):
    return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32) * scale).to(dtype)


def _write_blocks(case):
    return int(case["tokens"] / case["bs"] * 1.25) + 4


def _beams(rng, case, lens):
    """Block Tables of beams: a trunk, and branches that part from it towards the end."""
    bs, beams = case["bs"], case["beams"]
    rows, ids = len(lens) * beams, 0
    blocks = -(-lens // bs)
    tables = np.full((rows, int(blocks.max()) + 1), -1, dtype=np.int64)
    for r, n in enumerate(blocks):
        branch = np.arange(beams)  # which of the column's blocks each beam has
        for j in range(int(n) - 1, -1, -1):
            if branch.max() == 0:  # the trunk
                tables[r * beams:(r + 1) * beams, :j + 1] = ids + np.arange(j + 1)
                ids += j + 1
                break
            tables[r * beams:(r + 1) * beams, j] = ids + branch
            k = int(branch.max()) + 1
            ids += k
            branch = np.unique(rng.integers(0, max(1, k * 2 // 3), size=k)[branch], return_inverse=True)[1].reshape(-1)
    return tables, ids


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    op, hkv, d, bs, dtype = case["op"], case["hkv"], case["d"], case["bs"], DTYPES[case["dtype"]]
    if op == "write":
        t, hq = case["tokens"], case["hq"]
        # values of unequal size, as channels and heads have them
        size = torch.exp(torch.randn((2 * hkv, d), generator=gen, device="cuda"))
        if case["fused"]:
            qkv = _normal(gen, (t, (hq + 2 * hkv) * d), dtype)
            qkv[:, hq * d:] *= size.flatten().to(dtype)
            s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        else:
            s["k"], s["v"] = (_normal(gen, (t, hkv, d), dtype) * m.to(dtype) for m in size.chunk(2))
        blocks = _write_blocks(case)
        slots = rng.permutation(blocks * bs)[:t]
        slots[rng.random(t) < 0.02] = -1  # a padded batch
        s["slots"] = _i32(slots)
        s["all_slots"] = torch.arange(blocks * bs, dtype=torch.int32, device="cuda")
        s["k_cache"], s["v_cache"] = _cache(gen, blocks, case), _cache(gen, blocks, case)
        return s
    lens, rows = _lens(case)
    order = rng.permutation(len(lens))
    lens, rows = lens[order], rows[order]
    if op == "fork":
        beams = case["beams"]
        tables, used = _beams(np.random.default_rng(0), case, _lens(case)[0])  # as many pages for every seed
        tables = tables.reshape(len(lens), beams, -1)[order].reshape(len(lens) * beams, -1)
        pool = used + 2 * len(tables) + 16
        perm = rng.permutation(pool)
        s["tables"] = _i32(np.where(tables >= 0, perm[np.maximum(tables, 0)], -1))
        s["lens"] = _i32(np.repeat(lens, beams))
        parents = rng.integers(0, beams, size=(len(lens), beams)) + beams * np.arange(len(lens))[:, None]
        parents[rng.random(len(lens)) < 0.06] = -2  # a finished request gives its pages back
        s["parents"] = _i32(parents.reshape(-1))
        pinned = rng.random(pool) < 0.01  # pages that another part of the program holds
        pinned[perm[used:used + 2 * len(tables) + 8]] = False
        s["pinned"] = torch.from_numpy(pinned).cuda()
        s["num_blocks"] = pool
        s["caches"] = [_normal(gen, (pool, bs, hkv, d), dtype) for _ in range(2 * case["layers"])]
        return s
    s["lens"] = _i32(lens)
    tables, pool = _tables(rng, lens, bs)
    s["tables"] = _i32(tables)
    s["k_cache"], s["v_cache"] = _cache(gen, pool, case), _cache(gen, pool, case)
    s["scale"] = 1.0 / math.sqrt(d)
    s["host_lens"], s["host_rows"] = lens.tolist(), rows.tolist()  # what the program that made the batch knows
    if op == "decode":
        shape = (case["batch"], case["hq"], d)
        if case["q_len"] > 1:
            shape = shape[:1] + (case["q_len"],) + shape[1:]
        s["q"] = _normal(gen, shape, dtype, 2.0)
    else:
        s["q_start"] = _i32(np.concatenate([[0], np.cumsum(rows)]))
        s["max_q_len"] = int(rows.max())
        s["q"] = _normal(gen, (int(rows.sum()), case["hq"], d), dtype, 2.0)
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _write_plain(s):
    used = (s["slots"] >= 0).nonzero().squeeze(1)
    slots = s["slots"][used].long()
    out = []
    for cache, x in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        v = _values(*_unpack(cache, s["bs"], s["d"])).flatten(0, 1)
        v[slots] = _values(*_encode(x[used].float()))
        out.append(v.to(x.dtype))
    return tuple(out)


def _sequence(s, r):
    """K and V of sequence r as [kv head, token, d] in 32 bits."""
    n = s["host_lens"][r]
    blocks = s["tables"][r, :-(-n // s["bs"])].long()
    return [_values(*_unpack(c[blocks], s["bs"], s["d"])).flatten(0, 1)[:n].transpose(0, 1)
            for c in (s["k_cache"], s["v_cache"])]


def _attend_plain(s):
    hq, hkv, d = s["hq"], s["hkv"], s["d"]
    q = s["q"].float().reshape(-1, hkv, hq // hkv, d)
    out = torch.empty_like(q)
    at = 0
    for r, (n, rows) in enumerate(zip(s["host_lens"], s["host_rows"])):
        k, v = _sequence(s, r)
        last = n - rows + torch.arange(rows, device="cuda")  # the last key each query sees
        seen = (torch.arange(n, device="cuda")[None] <= last[:, None])[:, None]
        step = max(1, int(2e9 / (rows * (hq // hkv) * n)))  # heads at a time
        for h in range(0, hkv, step):
            x = q[at:at + rows, h:h + step].transpose(0, 1).flatten(1, 2)
            w = torch.matmul(x, k[h:h + step].transpose(1, 2)).mul_(s["scale"])
            w.view(-1, rows, hq // hkv, n).masked_fill_(~seen, -math.inf)
            top = w.amax(-1, keepdim=True)
            w = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
            total = w.sum(-1, keepdim=True)
            y = torch.matmul(w, v[h:h + step]) / torch.where(total == 0, torch.ones_like(total), total)
            out[at:at + rows, h:h + step] = y.view(-1, rows, hq // hkv, d).transpose(0, 1)
        at += rows
    return out.view(s["q"].shape).to(s["q"].dtype)


def _fork_plain(s):
    bs, tables, parents, num_blocks = s["bs"], s["tables"].long(), s["parents"].long(), s["num_blocks"]
    rows, width = len(parents), tables.shape[1]
    row = torch.arange(rows, device="cuda")
    live = parents >= 0
    length = torch.where(live, s["lens"].long()[parents.clamp_min(0)], 0)
    grow = torch.where(parents >= -1, 1, 0)
    have, want = (length + bs - 1) // bs, (length + grow + bs - 1) // bs
    col = torch.arange(width, device="cuda")[None]
    new = torch.where(col < have[:, None], tables[parents.clamp_min(0)], -1)
    count = torch.bincount(new[new >= 0], minlength=num_blocks)
    # a row that goes on inside a page has it to itself: the first such row, if no one else holds it
    writes = live & (grow > 0) & (length % bs != 0)
    tail = new.gather(1, (have - 1).clamp_min(0)[:, None])[:, 0].clamp_min(0)
    writers = torch.bincount(tail[writes], minlength=num_blocks)
    first = torch.full((num_blocks,), rows, device="cuda").scatter_reduce(
        0, torch.where(writes, tail, 0), torch.where(writes, row, rows), "amin")
    keeps = (first[tail] == row) & (count[tail] == writers[tail]) & ~s["pinned"][tail]
    copies = writes & ~keeps
    # pages in order of their number, to the rows in order: the copy's, then those of new tokens
    free = ((count == 0) & ~s["pinned"]).nonzero().squeeze(1)
    need = copies.long() + want - have
    start = torch.cumsum(need, 0) - need
    dst = free[start.clamp_max(len(free) - 1)]
    pairs = torch.where(copies[:, None], torch.stack([tail, dst], 1), -1)
    new = torch.where(copies[:, None] & (col == have[:, None] - 1), dst[:, None], new)
    fresh = (start + copies.long())[:, None] + col - have[:, None]
    new = torch.where((col >= have[:, None]) & (col < want[:, None]), free[fresh.clamp(0, len(free) - 1)], new)
    slot = new.gather(1, (length // bs).clamp_max(width - 1)[:, None]) * bs + (length % bs)[:, None]
    slots = torch.where(grow[:, None] > 0, slot, -1)
    left = (len(free) - need.sum()).reshape(1)
    moved = pairs[copies]
    for c in s["caches"]:
        c[moved[:, 1]] = c[moved[:, 0]]
    i32 = [x.to(torch.int32) for x in (new, length + grow, pairs, slots, left)]
    return (*i32, *s["caches"])


PLAIN = {"write": _write_plain, "decode": _attend_plain, "prefill": _attend_plain, "fork": _fork_plain}


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------
def _own(s):
    from paged_kv_cache_76_gb300 import ops
    op = s["op"]
    if op == "write":
        ops.quantize_and_cache(s["k"], s["v"], s["slots"], s["k_cache"], s["v_cache"])
        return ops.dequantize_kv4(s["k_cache"], s["v_cache"], s["all_slots"], s["d"], dtype=s["k"].dtype)
    if op == "decode":
        return ops.decode_kv4(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"])
    if op == "prefill":
        return ops.chunked_prefill_kv4(s["q"], s["q_start"], s["lens"], s["k_cache"], s["v_cache"], s["tables"],
                                       s["scale"], s["max_q_len"])
    tables, lens, pairs, slots, left = ops.fork_blocks(s["tables"], s["lens"], s["parents"], s["num_blocks"], s["bs"],
                                                       grow=1, pinned=s["pinned"])
    ops.copy_pages(s["caches"], pairs)
    return (tables, lens, pairs, slots, left, *s["caches"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# the definition in 64 bits
# --------------------------------------------------------------------------
def _numbers64(pages, bs, d):
    """What pages [n, heads, bytes] hold, [n, bs, heads, d] in 64 bits."""
    n, heads, size = pages.shape
    rows = pages[..., :bs * d // 2].reshape(n, heads, bs, d // 2)
    byte = pages[..., bs * d // 2:].reshape(n, heads, bs, d // 16).long()
    scale = torch.where(byte < 8, byte.double() * 2.0 ** -17,
                        (8 + byte % 8).double() * torch.exp2((byte // 8).double() - 18))
    out = torch.empty((n, heads, bs, d), dtype=torch.float64, device=pages.device)
    for k in range(2):
        c = (rows >> 4 * k) % 16
        mag, sign = (c % 8).double(), 1.0 - 2.0 * (c >= 8).double()
        mag = torch.where(mag < 4, mag / 2, torch.where(mag < 6, mag - 2, 2 * mag - 8))
        out[..., k::2] = sign * mag
    out *= torch.repeat_interleave(scale, 16, -1)
    return out.transpose(1, 2)


def _nearest64(x, grid):
    """Index of the nearest entry of an ascending grid; the even one where two are as near."""
    i = torch.searchsorted(grid, x).clamp(1, len(grid) - 1)
    below, above = x - grid[i - 1], grid[i] - x
    low = (below < above) | ((below == above) & (i % 2 == 1))
    return torch.where(low, i - 1, i)


def _write_exact(s):
    byte = torch.arange(TOP_SCALE + 1, device="cuda")
    scales = torch.where(byte < 8, byte.double() * 2.0 ** -17,
                         (8 + byte % 8).double() * torch.exp2((byte // 8).double() - 18))
    levels = torch.tensor(LEVELS, dtype=torch.float64, device="cuda")
    out = []
    for cache, x in ((s["k_cache"], s["k"]), (s["v_cache"], s["v"])):
        held = _numbers64(cache, s["bs"], s["d"]).flatten(0, 1).clone()
        g = x.double().reshape(-1, s["hkv"], s["d"] // 16, 16)
        scale = scales[_nearest64(g.abs().max(-1).values / 6, scales)][..., None]
        part = torch.where(scale > 0, g.abs() / scale, 0.0)
        v = (levels[_nearest64(part, levels)] * scale * torch.sign(g)).reshape(x.shape)
        for_slot = s["slots"].long()
        held[for_slot[for_slot >= 0]] = v[for_slot >= 0]
        out.append(held)
    return tuple(out)


def _attend_exact(s):
    hq, hkv, d, bs = s["hq"], s["hkv"], s["d"], s["bs"]
    group = hq // hkv
    q = s["q"].reshape(-1, hq, d)
    out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
    at = 0
    for r, (n, rows) in enumerate(zip(s["host_lens"], s["host_rows"])):
        blocks = s["tables"][r, :(n + bs - 1) // bs].long()
        for h in range(hkv):
            k, v = (_numbers64(c[blocks][:, h:h + 1], bs, d).reshape(-1, d)[:n] for c in (s["k_cache"], s["v_cache"]))
            for i in range(0, rows, 512):
                m = min(512, rows - i)
                x = q[at + i:at + i + m, h * group:(h + 1) * group].double() @ k.T * s["scale"]
                hidden = torch.arange(n, device="cuda") > (n - rows + i + torch.arange(m, device="cuda"))[:, None]
                x.masked_fill_(hidden[:, None], -math.inf)
                p = torch.nan_to_num(torch.softmax(x, -1))  # a query that sees nothing: zeros
                out[at + i:at + i + m, h * group:(h + 1) * group] = p @ v
        at += rows
    return out.view(s["q"].shape)


EXACT = {"write": _write_exact, "decode": _attend_exact, "prefill": _attend_exact}


def exact(case, seed):
    if case["op"] not in EXACT:  # whole numbers and copies: compared for equality
        return None
    return EXACT[case["op"]](prepare(case, seed))
