"""The 4-bit cache in 64 bits, for the tests: pages to numbers, numbers to the
nearest that a group can hold, and attention over them."""
import torch

LEVELS = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64)


def scale_values():
    """What each of the 256 scale bytes stands for."""
    b = torch.arange(256, dtype=torch.int16) << 7
    return b.view(torch.float16).double()


def numbers(cache, bs, d):
    """uint8 [n, heads, page] -> float64 [n, bs, heads, d]."""
    cache = cache.cpu()
    n, heads, page = cache.shape
    assert page == bs * (d // 2 + d // 16)
    codes = cache[:, :, :bs * d // 2].reshape(n, heads, bs, d // 2).long()
    scales = scale_values()[cache[:, :, bs * d // 2:].reshape(n, heads, bs, d // 16).long()]
    x = torch.empty(n, heads, bs, d, dtype=torch.float64)
    for k in range(2):
        c = codes >> (4 * k) & 15
        x[..., k::2] = torch.where(c < 8, LEVELS[c % 8], -LEVELS[c % 8])
    return (x.unflatten(-1, (d // 16, 16)) * scales[..., None]).flatten(-2).transpose(1, 2)


def nearest(x, grid):
    """Index in an ascending grid; of two as near, the even one."""
    d = (x.clamp(max=float(grid[-1]))[..., None] - grid).abs()  # far above the grid every distance rounds to the same
    best = d.min(-1, keepdim=True).values
    i = torch.arange(len(grid))
    cand = torch.where(d == best, i + (i % 2) * 1000, 10 ** 6)
    return cand.argmin(-1)


def quantized(x):
    """float64 [..., d]: what the cache holds of it, and the scale bytes [..., d / 16]."""
    g = x.double().cpu().unflatten(-1, (-1, 16))
    top = g.abs().amax(-1)
    grid = scale_values()[:0xE3]
    byte = nearest(torch.nan_to_num(top, posinf=0.0) / 6, grid)
    s = grid[byte][..., None]
    y = torch.where(s > 0, g.abs() / torch.where(s > 0, s, 1.0), 0.0)
    v = torch.sign(g) * LEVELS[nearest(torch.nan_to_num(y), LEVELS)] * s
    bad = ~g.isfinite().all(-1)
    byte = torch.where(bad, 0xFF, byte)
    v = torch.where(bad[..., None], float("nan"), v)
    return v.flatten(-2), byte


def attend(q, k, v, scale, seen):
    """q [rows, d], k, v [n, d], seen [rows, n], float64: outputs, and per output the size that errors are counted in
    (weights' errors times |v|)."""
    x = q @ k.T * scale
    x = x.masked_fill(~seen, -float("inf"))
    empty = ~seen.any(-1)
    p = torch.softmax(x, -1)
    p[empty] = 0.0
    v0 = torch.where(seen.any(0)[:, None], v, 0.0)
    out = p @ v0
    # a row that sees a token that is not a number is none
    return out, p @ v0.abs()
