"""Cases of the operators for caches whose slot order is not the position order.

Five operators of the library, each in its plain form (elementary torch
operations in 32 bits, rounded once at the end) and as the library's call:

* ``rope``: per-head norm of queries and keys, rotary positions (one axis or
  time/height/width), queries out, keys and values into the paged cache
  (``ops.norm_rope_and_cache``);
* ``tree``: attention of a tree of drafted tokens over the paged cache
  (``ops.verify_tree``);
* ``accumulate``: decode that also adds each cached token's attention weight
  to its score (``ops.decode_accumulate``);
* ``select``: the tokens a budget keeps: the first, the last, and the best
  scored between (``ops.evict_select``);
* ``compact``: the kept tokens moved to the front of their sequence, in place
  (``ops.compact_kv``): after an eviction, or after a tree's accepted path.

Sizes follow the workloads of this repository (32/8, 64/8 and 28/4 heads of
128, 16-token blocks, contexts of hundreds to 131072 tokens) and odd ones
around them.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
GOLDEN = 0.6180339887498949


# --------------------------------------------------------------------------
# cases
# --------------------------------------------------------------------------
def listed():
    return [
        # one decode step's new tokens of a batch: a launch of a few microseconds
        dict(name="rope_decode_64", op="rope", tokens=64, hq=32, hkv=8, d=128, rot=128, axes=1, norm=True,
             fused=False, interleaved=False, bs=16, dtype="bf16", max_pos=131072),
        # one prefill step, q/k/v as views of a fused projection's rows
        dict(name="rope_prefill_8192", op="rope", tokens=8192, hq=32, hkv=8, d=128, rot=128, axes=1, norm=True,
             fused=True, interleaved=False, bs=16, dtype="bf16", max_pos=131072),
        # an image's tokens: three position axes, no norm, an odd count
        dict(name="rope_axes_4095", op="rope", tokens=4095, hq=28, hkv=4, d=128, rot=128, axes=3, norm=False,
             fused=True, interleaved=False, bs=16, dtype="fp16", max_pos=32768),
        # few requests, small ragged trees, odd contexts: latency
        dict(name="tree_small", op="tree", batch=4, lo=301, hi=1501, nlo=3, nhi=9, hq=28, hkv=4, d=128, bs=16,
             dtype="bf16"),
        # a serving batch verifying 26 to 60 drafted tokens a request
        dict(name="tree_batch_64", op="tree", batch=64, lo=509, hi=4079, nlo=26, nhi=60, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # long contexts, 16 nodes: the keys have to be split over the GPU
        dict(name="tree_long", op="tree", batch=8, lo=32768, hi=131009, nlo=16, nhi=16, hq=64, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # a decode step that keeps score
        dict(name="accumulate_64", op="accumulate", batch=64, lo=509, hi=4079, hq=32, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # the same over long contexts
        dict(name="accumulate_long", op="accumulate", batch=8, lo=32768, hi=131009, hq=64, hkv=8, d=128, bs=16,
             dtype="bf16"),
        # a serving batch cut to a budget of 1024 tokens
        dict(name="select_64", op="select", batch=64, lo=509, hi=4079, hkv=8, sink=4, heavy=508, recent=512),
        # long contexts cut to 8192
        dict(name="select_long", op="select", batch=8, lo=32768, hi=131009, hkv=8, sink=4, heavy=4092, recent=4096),
        # the accepted paths of a batch of trees, one list for all heads
        dict(name="compact_paths_64", op="compact", batch=64, lo=509, hi=4079, keep=8, window=60, per_head=False,
             scored=False, hkv=8, d=128, bs=16, dtype="bf16"),
        # long contexts after an eviction: every head keeps its own 8192 tokens, their scores follow
        dict(name="compact_evicted", op="compact", batch=8, lo=32768, hi=131009, keep=8192, window=0, per_head=True,
             scored=True, hkv=8, d=128, bs=16, dtype="bf16"),
    ]


def draw(rng):
    op = rng.choice(["rope", "tree", "accumulate", "select", "compact"])
    log = lambda a, b: int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))  # noqa: E731
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    d = rng.choice([128, 128, 64])
    heads = [(32, 8), (28, 4), (64, 8), (16, 2), (8, 1), (12, 12)] if d == 128 else [(28, 4), (64, 8), (16, 2), (12, 12)]
    hq, hkv = rng.choice(heads)
    bs = rng.choice([4, 8, 16, 16, 32])
    if op == "rope":
        return dict(op=op, tokens=log(1, 8192), hq=hq, hkv=hkv, d=d, rot=rng.choice([d, d, d // 2, 48]),
                    axes=rng.choice([1, 1, 3]), norm=rng.random() < 0.7, fused=rng.random() < 0.5,
                    interleaved=rng.random() < 0.3, bs=bs, dtype=dtype, max_pos=log(1024, 131072))
    if op == "select":
        batch = log(1, 96)
        hi = log(100, min(131072, 2000000 // batch))
        heavy = log(1, max(2, hi // 3))
        return dict(op=op, batch=batch, lo=max(1, hi // rng.choice([2, 8, 50])), hi=hi, hkv=hkv,
                    sink=rng.choice([0, 1, 4]), heavy=heavy, recent=rng.choice([1, 64, heavy]))
    batch = log(1, 64)
    hi = log(40, min(131072, 400000 // batch))
    lo = max(1, hi // rng.choice([2, 8, 50]))
    if op == "tree":
        nhi = log(1, 64)
        return dict(op=op, batch=batch, lo=lo, hi=hi, nlo=max(1, nhi // 2), nhi=nhi, hq=hq, hkv=hkv, d=d, bs=bs,
                    dtype=dtype)
    if op == "accumulate":
        return dict(op=op, batch=batch, lo=lo, hi=hi, hq=hq, hkv=hkv, d=d, bs=bs, dtype=dtype)
    if rng.random() < 0.5:
        window = log(1, min(64, lo))
        return dict(op=op, batch=batch, lo=lo, hi=hi, keep=log(1, window), window=window, per_head=False,
                    scored=False, hkv=hkv, d=d, bs=bs, dtype=dtype)
    return dict(op=op, batch=batch, lo=lo, hi=hi, keep=log(1, max(2, hi // 2)), window=0, per_head=True,
                scored=rng.random() < 0.7, hkv=hkv, d=d, bs=bs, dtype=dtype)


def _spread(n, lo, hi, phase):
    """n whole numbers over [lo, hi], the same for every seed (a low-discrepancy sequence)."""
    return (lo + np.floor((hi - lo + 1) * ((np.arange(n) * GOLDEN + phase) % 1.0))).astype(np.int64)


def _lens(case):
    """Context lengths of the batch; a tree's nodes are counted in."""
    hist = _spread(case["batch"], case["lo"], case["hi"], 0.5)
    if case["op"] != "tree":
        return hist, None
    nodes = _spread(case["batch"], case["nlo"], case["nhi"], 0.25)
    return hist + nodes, nodes


def work(case):
    op = case["op"]
    if op == "rope":
        t, hq, hkv, d = case["tokens"], case["hq"], case["hkv"], case["d"]
        elems = t * (hq + 2 * hkv) * d
        pos = 4 * t * (case["axes"] + 1)
        table = 4 * case["rot"] * min(t * case["axes"], case["max_pos"])
        return {"bytes": 4 * elems + pos + table, "flops": t * (hq + hkv) * (4 * d * case["norm"] + 3 * case["rot"])}
    lens, nodes = _lens(case)
    hkv, total = case["hkv"], int(lens.sum())
    if op == "select":
        kept = int(np.minimum(lens, case["sink"] + case["heavy"] + case["recent"]).sum())
        return {"bytes": 4 * hkv * (total + kept), "flops": hkv * total}
    d = case["d"]
    if op == "compact":
        kept = int(np.minimum(lens - _base(case, lens), case["keep"]).sum())
        per_token = 8 * d + (4 if case["per_head"] else 0) + (8 if case["scored"] else 0)
        return {"bytes": hkv * kept * per_token, "flops": 0}
    kv = 4 * total * hkv * d
    rows = int((nodes if nodes is not None else np.ones_like(lens)).sum()) * case["hq"]
    flops = 4 * int(((nodes if nodes is not None else 1) * lens).sum()) * case["hq"] * d
    extra = 8 * total * hkv if op == "accumulate" else 0
    return {"bytes": kv + 4 * rows * d + 4 * total // case["bs"] + extra, "flops": flops}


# --------------------------------------------------------------------------
# inputs
# --------------------------------------------------------------------------
def _sections(case):
    half = case["rot"] // 2
    if case["axes"] == 1:
        return None
    t = half // 4 // 8 * 8
    h = (half - t) // 2
    return (t, h, half - t - h)


def _base(case, lens):
    """First token a compaction may move: the draft's first, or the sequence's."""
    return lens - np.minimum(case["window"], lens) if case["window"] else np.zeros_like(lens)


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


def _pool(gen, pool, case):
    shape = (pool, case["bs"], case["hkv"], case["d"])
    dtype = DTYPES[case["dtype"]]
    return (torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen),
            torch.empty(shape, dtype=dtype, device="cuda").normal_(generator=gen))


def _scores(gen, rows, hkv, lens, score_rows):
    """Accumulated weights as a run of decode steps leaves them: a heavy tail,
    equal values among them, zero behind each sequence."""
    width = int(lens.max() + 15) // 16 * 16
    s = torch.randn((rows, hkv, width), generator=gen, device="cuda", dtype=torch.float32).mul_(2.0).exp_()
    s = torch.round(s * 4096.0) / 4096.0
    held = torch.zeros(rows, dtype=torch.int64, device="cuda")
    held[score_rows.long()] = torch.from_numpy(lens).cuda()
    s.masked_fill_(torch.arange(width, device="cuda")[None, None] >= held[:, None, None], 0.0)
    return s


def _table_of_angles(max_pos, rot):
    """cos | sin of position * 10000^(-2j/rot), [max_pos, rot], computed in 64 bits."""
    j = torch.arange(rot // 2, device="cuda", dtype=torch.float64)
    a = torch.arange(max_pos, device="cuda", dtype=torch.float64)[:, None] * torch.pow(10000.0, -2.0 * j / rot)[None]
    return torch.cat([a.cos(), a.sin()], 1).to(torch.float32)


def prepare(case, seed):
    rng = np.random.default_rng(seed)
    gen = torch.Generator(device="cuda").manual_seed(seed)
    s = dict(case)
    if case["op"] == "rope":
        t, hq, hkv, d, dtype = case["tokens"], case["hq"], case["hkv"], case["d"], DTYPES[case["dtype"]]
        if case["fused"]:
            qkv = _normal(gen, (t, (hq + 2 * hkv) * d), dtype)
            s["q"] = qkv[:, :hq * d].unflatten(1, (hq, d))
            s["k"] = qkv[:, hq * d:(hq + hkv) * d].unflatten(1, (hkv, d))
            s["v"] = qkv[:, (hq + hkv) * d:].unflatten(1, (hkv, d))
        else:
            s["q"], s["k"], s["v"] = (_normal(gen, (t, h, d), dtype) for h in (hq, hkv, hkv))
        s["qw"], s["kw"] = ((_normal(gen, (d,), dtype, 0.1) + 1).to(dtype) for _ in range(2)) if case["norm"] \
            else (None, None)
        pos = rng.integers(0, case["max_pos"], size=(case["axes"], t))
        s["positions"] = _i32(pos if case["axes"] > 1 else pos[0])
        s["cos_sin"] = _table_of_angles(case["max_pos"], case["rot"])
        s["sections"] = _sections(case)
        blocks = int(t / case["bs"] * 1.25) + 4
        slots = rng.permutation(blocks * case["bs"])[:t]
        slots[rng.random(t) < 0.02] = -1  # a padded batch
        s["slots"] = _i32(slots)
        s["k_cache"], s["v_cache"] = _pool(gen, blocks, case)
        return s
    lens, nodes = _lens(case)
    order = rng.permutation(len(lens))
    lens = lens[order]
    s["lens"] = _i32(lens)
    if case["op"] in ("select", "accumulate") or case["op"] == "compact" and case["scored"]:
        s["score_rows"] = _i32(rng.permutation(case["batch"] + 2)[:case["batch"]])
        s["scores"] = _scores(gen, case["batch"] + 2, case["hkv"], lens, s["score_rows"])
    if case["op"] == "select":
        return s
    tables, pool = _tables(rng, lens, case["bs"])
    s["tables"] = _i32(tables)
    s["k_cache"], s["v_cache"] = _pool(gen, pool, case)
    s["scale"] = 1.0 / math.sqrt(case["d"])
    if case["op"] == "accumulate":
        s["q"] = _normal(gen, (case["batch"], case["hq"], case["d"]), DTYPES[case["dtype"]], 2.0)
        s["scores_out"] = torch.zeros_like(s["scores"])
    elif case["op"] == "tree":
        nodes = nodes[order]
        start = np.concatenate([[0], np.cumsum(nodes)])
        n_max = int(nodes.max())
        masks = np.zeros((len(lens), n_max), dtype=np.uint64)
        for i in range(n_max):  # node i's parent is an earlier node, or the context
            parent = rng.integers(max(-1, i - 6), i, size=len(lens)) if i else np.full(len(lens), -1)
            above = np.where(parent >= 0, masks[np.arange(len(lens)), np.maximum(parent, 0)], np.uint64(0))
            masks[:, i] = above | np.uint64(1 << i)
        masks[::4, -1] = 0  # a padding node: it sees the context alone, and no node sees it
        keep = np.arange(n_max)[None] < nodes[:, None]
        s["q_start"] = _i32(start)
        s["nodes"] = _i32(nodes)
        s["mask"] = torch.from_numpy(masks[keep].view(np.int64)).cuda()
        s["max_q_len"] = n_max
        s["q"] = _normal(gen, (int(start[-1]), case["hq"], case["d"]), DTYPES[case["dtype"]], 2.0)
        # where each row of q stands in a padded batch
        s["row"] = torch.from_numpy(np.nonzero(keep.reshape(-1))[0]).cuda()
    else:
        base = _base(case, lens)
        room = lens - base
        heads = case["hkv"] if case["per_head"] else 1
        width = int(room.max())
        tag = torch.rand((case["batch"], heads, width), generator=gen, device="cuda")
        tag.masked_fill_(torch.arange(width, device="cuda")[None, None] >= torch.from_numpy(room).cuda()[:, None, None],
                         2.0)
        count = np.minimum(room, case["keep"])
        keep = torch.argsort(tag, -1)[..., :int(count.max())]
        behind = torch.arange(keep.shape[-1], device="cuda")[None, None] >= torch.from_numpy(count).cuda()[:, None, None]
        keep = keep.masked_fill(behind, 1 << 30).sort(-1).values
        s["keep"] = keep.masked_fill(behind, -1).to(torch.int32).contiguous()
        s["keep_lens"] = _i32(count)
        s["base"] = _i32(base) if case["window"] else None
    return s


# --------------------------------------------------------------------------
# the plain forms
# --------------------------------------------------------------------------
def _rotate_plain(x, s, weight):
    x = x.float()
    if weight is not None:
        x = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6) * weight.float()
    rot, half = s["rot"], s["rot"] // 2
    pos = s["positions"].long()
    if s["sections"] is None:
        cs = s["cos_sin"][pos]
        cos, sin = cs[:, :half], cs[:, half:]
    else:
        axis = torch.repeat_interleave(torch.arange(3, device=x.device), torch.tensor(s["sections"], device=x.device))
        at = pos[axis].T  # [tokens, half]
        j = torch.arange(half, device=x.device)[None]
        cos, sin = s["cos_sin"][at, j], s["cos_sin"][at, j + half]
    cos, sin = cos[:, None], sin[:, None]
    if s["interleaved"]:
        a, b = x[..., 0:rot:2], x[..., 1:rot:2]
        turned = torch.stack([a * cos - b * sin, b * cos + a * sin], -1).flatten(-2)
    else:
        a, b = x[..., :half], x[..., half:rot]
        turned = torch.cat([a * cos - b * sin, b * cos + a * sin], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _rope_plain(s):
    dtype = s["q"].dtype
    out = _rotate_plain(s["q"], s, s["qw"]).to(dtype)
    k = _rotate_plain(s["k"], s, s["kw"]).to(dtype)
    used = (s["slots"] >= 0).nonzero().squeeze(1)
    slots = s["slots"][used].long()
    s["k_cache"].view(-1, s["hkv"], s["d"])[slots] = k[used]
    s["v_cache"].view(-1, s["hkv"], s["d"])[slots] = s["v"][used]
    return out, s["k_cache"], s["v_cache"]


def _gathered(s):
    """Every sequence's K and V in 32 bits, [batch, kv head, token, d]: zero behind the sequence."""
    bs, n = s["bs"], s["tables"].shape[1] * s["bs"]
    t = torch.arange(n, device="cuda")
    slot = s["tables"].long().clamp_min(0)[:, t // bs] * bs + t % bs
    held = (t[None] < s["lens"][:, None])
    k, v = (c.view(-1, s["hkv"], s["d"])[slot].permute(0, 2, 1, 3).float().masked_fill_(~held[:, None, :, None], 0.0)
            for c in (s["k_cache"], s["v_cache"]))
    return k, v, t, held


def _attend_plain(q, k, v, seen, scale):
    """q [batch, kv head, rows, d]; seen [batch, 1, rows, tokens]: outputs and weights, zero where a row sees nothing."""
    w = torch.matmul(q, k.transpose(-1, -2)).mul_(scale).masked_fill_(~seen, -math.inf)
    top = w.amax(-1, keepdim=True)
    w = w.sub_(torch.where(top == -math.inf, torch.zeros_like(top), top)).exp_()
    total = w.sum(-1, keepdim=True)
    w = w.div_(torch.where(total == 0, torch.ones_like(total), total))
    return torch.matmul(w, v), w


def _tree_plain(s):
    k, v, t, held = _gathered(s)
    b, n, hq, hkv, d = len(s["lens"]), s["max_q_len"], s["hq"], s["hkv"], s["d"]
    g = hq // hkv
    q = torch.zeros((b * n, hq, d), device="cuda")
    q[s["row"]] = s["q"].float()
    q = q.view(b, n, hkv, g, d).permute(0, 2, 1, 3, 4).reshape(b, hkv, n * g, d)
    mask = torch.zeros(b * n, dtype=torch.int64, device="cuda")
    mask[s["row"]] = s["mask"]
    node = t[None] - (s["lens"] - s["nodes"])[:, None]  # < 0: the context before the draft
    bit = (mask.view(b, n, 1) >> node.clamp(0, 63)[:, None]) & 1
    seen = ((node < 0)[:, None] | (bit == 1)) & held[:, None]
    seen = seen[:, :, None].expand(b, n, g, len(t)).reshape(b, 1, n * g, len(t))
    out, _ = _attend_plain(q, k, v, seen, s["scale"])
    out = out.view(b, hkv, n, g, d).permute(0, 2, 1, 3, 4).reshape(b * n, hq, d)
    return out[s["row"]].to(s["q"].dtype)


def _accumulate_plain(s):
    k, v, t, held = _gathered(s)
    b, hq, hkv, d = len(s["lens"]), s["hq"], s["hkv"], s["d"]
    q = s["q"].float().view(b, hkv, hq // hkv, d)
    out, w = _attend_plain(q, k, v, held[:, None, None], s["scale"])
    width = min(s["scores"].shape[-1], len(t))
    rows = s["score_rows"].long()
    new = s["scores"][rows][..., :width] + w.sum(2)[..., :width]
    old = s["scores_out"][rows][..., :width]
    s["scores_out"][rows, :, :width] = torch.where(held[:, None, :width], new, old)
    return out.reshape(b, hq, d).to(s["q"].dtype), s["scores_out"]


def _select_plain(s):
    budget = s["sink"] + s["heavy"] + s["recent"]
    scores = s["scores"][s["score_rows"].long()]
    b, hkv, width = scores.shape
    t = torch.arange(width, device="cuda")[None, None]
    lens = s["lens"].long()[:, None, None]
    always = ((t < s["sink"]) | (t >= lens - s["recent"])) & (t < lens)
    ranked = scores.masked_fill(always | (t >= lens), -math.inf)
    best = torch.sort(ranked, dim=-1, descending=True, stable=True).indices[..., :min(s["heavy"], width)]
    chosen = torch.zeros((b, hkv, width), dtype=torch.bool, device="cuda").scatter_(-1, best, True)
    chosen = (chosen | always | (lens <= budget)) & (t < lens)
    at = torch.where(chosen, t, torch.full_like(t, width)).sort(-1).values
    at = torch.nn.functional.pad(at, (0, max(0, budget - width)), value=width)[..., :budget]
    keep = torch.where(at == width, torch.full_like(at, -1), at).to(torch.int32)
    return keep, s["lens"].clamp_max(budget).to(torch.int32)


def _compact_plain(s):
    bs, hkv, d = s["bs"], s["hkv"], s["d"]
    keep = s["keep"].long().expand(-1, hkv, -1)
    i = torch.arange(keep.shape[-1], device="cuda")
    base = s["base"].long()[:, None, None] if s["base"] is not None else 0
    used = (i[None, None] < s["keep_lens"][:, None, None]).expand(keep.shape)
    r = torch.arange(len(s["lens"]), device="cuda")[:, None, None].expand(keep.shape)[used]
    h = torch.arange(hkv, device="cuda")[None, :, None].expand(keep.shape)[used]
    src, dst = (keep + base)[used], (i[None, None] + base).expand(keep.shape)[used]
    tables = s["tables"].long()
    src_slot, dst_slot = (tables[r, x // bs] * bs + x % bs for x in (src, dst))
    flat_k, flat_v = (c.view(-1, hkv, d) for c in (s["k_cache"], s["v_cache"]))
    flat_k[dst_slot, h] = flat_k[src_slot, h]
    flat_v[dst_slot, h] = flat_v[src_slot, h]
    if not s["scored"]:
        return s["k_cache"], s["v_cache"]
    rows = s["score_rows"].long()
    moved = s["scores"][rows[r], h, src]
    t = torch.arange(s["scores"].shape[-1], device="cuda")[None, None]
    first = (s["base"].long() if s["base"] is not None else 0) + s["keep_lens"].long()
    behind = (t >= first[:, None, None]) & (t < s["lens"].long()[:, None, None])
    s["scores"][rows] = s["scores"][rows].masked_fill(behind, 0.0)
    s["scores"][rows[r], h, dst] = moved
    return s["k_cache"], s["v_cache"], s["scores"]


PLAIN = {"rope": _rope_plain, "tree": _tree_plain, "accumulate": _accumulate_plain, "select": _select_plain,
         "compact": _compact_plain}


# --------------------------------------------------------------------------
# the library's calls
# --------------------------------------------------------------------------
def _own(s):
    from paged_kv_cache_76_gb300 import ops
    op = s["op"]
    if op == "rope":
        out = ops.norm_rope_and_cache(s["q"], s["k"], s["v"], s["positions"], s["cos_sin"], s["slots"], s["k_cache"],
                                      s["v_cache"], q_weight=s["qw"], k_weight=s["kw"], eps=1e-6,
                                      sections=s["sections"], interleaved=s["interleaved"])
        return out, s["k_cache"], s["v_cache"]
    if op == "tree":
        return ops.verify_tree(s["q"], s["q_start"], s["mask"], s["lens"], s["k_cache"], s["v_cache"], s["tables"],
                               s["scale"], s["max_q_len"])
    if op == "accumulate":
        return ops.decode_accumulate(s["q"], s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["scale"],
                                     s["scores"], score_rows=s["score_rows"], scores_out=s["scores_out"])
    if op == "select":
        return ops.evict_select(s["scores"], s["lens"], s["sink"], s["heavy"], s["recent"],
                                score_rows=s["score_rows"])
    ops.compact_kv(s["k_cache"], s["v_cache"], s["tables"], s["lens"], s["keep"], s["keep_lens"], base=s["base"],
                   scores=s.get("scores"), score_rows=s.get("score_rows"))
    return (s["k_cache"], s["v_cache"], s["scores"]) if s["scored"] else (s["k_cache"], s["v_cache"])


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# --------------------------------------------------------------------------
# the definition in 64 bits, one sequence (or one pair of a head) at a time
# --------------------------------------------------------------------------
def _sequence(s, r):
    """K and V of sequence r as [kv head, token, d] in 64 bits."""
    n = int(s["lens"][r])
    blocks = s["tables"][r, :-(-n // s["bs"])].long()
    return [c[blocks].flatten(0, 1)[:n].double().transpose(0, 1) for c in (s["k_cache"], s["v_cache"])]


def _softmax64(x):
    e = torch.exp(x - x.max(-1, keepdim=True).values)
    return e / e.sum(-1, keepdim=True)


def _rope_exact(s):
    half, rot = s["rot"] // 2, s["rot"]
    pos = s["positions"].long().reshape(s["axes"], -1)
    table = s["cos_sin"].double()
    sections = s["sections"] or (half,)
    axis = [a for a, n in enumerate(sections) for _ in range(n)]
    outs = []
    for x, w in ((s["q"], s["qw"]), (s["k"], s["kw"])):
        x = x.double().clone()
        if w is not None:
            x /= ((x ** 2).sum(-1, keepdim=True) / s["d"] + 1e-6).sqrt()
            x *= w.double()
        y = x.clone()
        for j in range(half):
            lo, hi = (2 * j, 2 * j + 1) if s["interleaved"] else (j, j + half)
            z = torch.complex(x[..., lo], x[..., hi])
            turn = torch.complex(table[pos[axis[j]], j], table[pos[axis[j]], half + j])
            z = z * turn[:, None]
            y[..., lo], y[..., hi] = z.real, z.imag
        outs.append(y)
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    for t, slot in enumerate(s["slots"].tolist()):
        if slot >= 0:
            kc[slot // s["bs"], slot % s["bs"]] = outs[1][t]
            vc[slot // s["bs"], slot % s["bs"]] = s["v"][t].double()
    return outs[0], kc, vc


def _tree_exact(s):
    start, out = s["q_start"].tolist(), torch.zeros(s["q"].shape, dtype=torch.float64, device="cuda")
    g = s["hq"] // s["hkv"]
    for r in range(len(start) - 1):
        k, v = _sequence(s, r)
        n = start[r + 1] - start[r]
        hist = k.shape[1] - n
        bits = s["mask"][start[r]:start[r + 1], None].expand(n, n).clone()
        for j in range(n):
            bits[:, j] = (bits[:, j] >> j) & 1
        q = s["q"][start[r]:start[r + 1]].double()
        for h in range(s["hq"]):
            x = q[:, h] @ k[h // g].T * s["scale"]
            x[:, hist:][bits == 0] = -math.inf
            p = torch.nan_to_num(_softmax64(x)) if hist == 0 else _softmax64(x)
            out[start[r]:start[r + 1], h] = p @ v[h // g]
    return out


def _accumulate_exact(s):
    g = s["hq"] // s["hkv"]
    out, scores = s["q"].double().clone(), s["scores_out"].double().clone()
    for r, row in enumerate(s["score_rows"].tolist()):
        k, v = _sequence(s, r)
        n = k.shape[1]
        scores[row, :, :n] = s["scores"][row, :, :n].double()
        for h in range(s["hq"]):
            p = _softmax64(k[h // g] @ s["q"][r, h].double() * s["scale"])
            out[r, h] = p @ v[h // g]
            scores[row, h // g, :n] += p
    return out, scores


def _compact_exact(s):
    kc, vc = s["k_cache"].double(), s["v_cache"].double()
    scored = s["scored"]
    scores = s["scores"].double() if scored else None
    bs, tables = s["bs"], s["tables"].long()
    for r, n in enumerate(s["keep_lens"].tolist()):
        first = int(s["base"][r]) if s["base"] is not None else 0
        for h in range(s["hkv"]):
            src = s["keep"][r, h if s["per_head"] else 0, :n].long() + first
            dst = torch.arange(first, first + n, device="cuda")
            for new, old in ((kc, s["k_cache"]), (vc, s["v_cache"])):
                new[tables[r, dst // bs], dst % bs, h] = old[tables[r, src // bs], src % bs, h].double()
            if scored:
                row = int(s["score_rows"][r])
                scores[row, h, first + n:int(s["lens"][r])] = 0
                scores[row, h, first:first + n] = s["scores"][row, h, src].double()
    return (kc, vc, scores) if scored else (kc, vc)


EXACT = {"rope": _rope_exact, "tree": _tree_exact, "accumulate": _accumulate_exact, "compact": _compact_exact}


def exact(case, seed):
    if case["op"] not in EXACT:  # whole numbers: compared for equality
        return None
    return EXACT[case["op"]](prepare(case, seed))
