"""pa_fork_blocks row by row on the host, for the tests: who holds which block is
kept as a list of holders per block."""


def fork(tables, lens, parents, grow, num_blocks, bs, width, max_grow, pinned=()):
    """Lists in, (tables, lens, pairs, slots, num_free) out, as lists."""
    pinned = set(pinned)
    rows = []  # per new row: (blocks it goes on from, its length, growth), or None
    for p, g in zip(parents, grow):
        if p < -1 or p >= len(tables) or not 0 <= g <= max_grow:
            rows.append(None)
            continue
        n = lens[p] if p >= 0 else 0
        if n < 0 or (p >= 0 and n > len(tables[p]) * bs) or -(-(n + g) // bs) > width:
            rows.append(None)
            continue
        rows.append((list(tables[p][:-(-n // bs)]) if p >= 0 else [], n, g))
    holders = {}
    for i, row in enumerate(rows):
        for j, b in enumerate(row[0] if row else []):
            inside = row[2] > 0 and row[1] % bs != 0 and j == len(row[0]) - 1
            holders.setdefault(b, []).append((i, inside))
    free = [b for b in range(num_blocks) if b not in holders and b not in pinned]
    total = len(free)
    out = []
    for i, row in enumerate(rows):
        if row is None:
            out.append(([], 0, (-1, -1), []))
            continue
        blocks, n, g = row
        pair = (-1, -1)
        if g > 0 and n % bs != 0 and 0 <= blocks[-1] < num_blocks:
            b = blocks[-1]
            alone = all(inside for _, inside in holders[b]) and b not in pinned
            if not (alone and holders[b][0][0] == i):
                if not free:
                    return refused(len(rows), width, max_grow, total)
                pair = (b, free.pop(0))
                blocks[-1] = pair[1]
        while len(blocks) * bs < n + g:
            if not free:
                return refused(len(rows), width, max_grow, total)
            blocks.append(free.pop(0))
        slots = [blocks[(n + t) // bs] * bs + (n + t) % bs if 0 <= blocks[(n + t) // bs] < num_blocks else -1
                 for t in range(g)]
        out.append((blocks, n + g, pair, slots))

    def pad(x, n):
        return x + [-1] * (n - len(x))
    return ([pad(b, width) for b, _, _, _ in out], [n for _, n, _, _ in out], [list(p) for _, _, p, _ in out],
            [pad(s, max_grow) for _, _, _, s in out], len(free))


def refused(rows, width, max_grow, total):
    return [[-1] * width] * rows, [0] * rows, [[-1, -1]] * rows, [[-1] * max_grow] * rows, total
