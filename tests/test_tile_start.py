"""The two query tiles of the tensor-core prefills share every K stage, and tile B
begins once tile A's first P is there.  What B waits on has to stay passed until
B looks, however late its queries come: a barrier tells one phase from the next
by its parity alone.

The kernels' start is followed here on the host, step by step as far as either
tile can go; the sources are read for the barrier that B waits on."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "paged_kv_cache_76_gb300", "csrc")
KERNELS = {"attn_tc.cu": ("kKStages", "kVStages"), "kv4_prefill.cu": ("kStages", "kStages")}


class Barrier:
    """One arrival a phase; a wait passes once the phase of its parity is over, by the parity of the phase under way."""

    def __init__(self):
        self.phase = 0

    def arrive(self):
        self.phase += 1

    def passed(self, parity):
        return self.phase % 2 != parity


def ends(tiles, k_stages, v_stages, late, own):
    """Do both tiles come to their end when B's queries are there after A's first `late` P?  Without `own` B waits on
    A's P barrier of even key tiles."""
    p_even, begun = Barrier(), Barrier()
    s = [0, 0]         # key tiles whose S each has issued: a K stage is free again when both have
    p = [0, 0]         # ... whose P is there, and its P.V issued: so is a V stage
    started = False
    while True:
        moved = False
        if not started and p[0] >= min(late, tiles) and (begun if own else p_even).passed(0):
            started = moved = True
        for x in (0, 1):
            if x == 1 and not started:
                continue
            if s[x] < tiles and s[x] - min(s) < k_stages and s[x] - p[x] < 2:
                s[x] += 1
                moved = True
            if p[x] < s[x] and p[x] - min(p) < v_stages:
                if x == 0 and p[0] % 2 == 0:
                    p_even.arrive()
                if x == 0 and p[0] == 0:
                    begun.arrive()
                p[x] += 1
                moved = True
        if p == [tiles, tiles]:
            return True
        if not moved:
            return False


@pytest.mark.parametrize("kernel", KERNELS)
def test_tile_b_begins_however_late_it_is(kernel):
    text = open(os.path.join(CSRC, kernel)).read()
    k, v = (int(re.search(r"constexpr int %s = (\d+);" % n, text).group(1)) for n in KERNELS[kernel])
    cases = [(tiles, late) for tiles in range(1, 12) for late in range(8)
             if late <= min(tiles, k, v)]  # as far as A comes without B
    assert all(ends(tiles, k, v, late, True) for tiles, late in cases)
    assert not all(ends(tiles, k, v, late, False) for tiles, late in cases)


@pytest.mark.parametrize("kernel", KERNELS)
def test_what_tile_b_waits_on_is_passed_once(kernel):
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, kernel)).read())
    waits = re.findall(r"x == 1[^;]*mbar_wait\(bar\((\w+)\), 0\)", text)
    assert len(waits) == 1
    name = waits[0]
    arrivals = re.findall(r"[^;{}]*mbar_arrive\(bar\(%s\b[^;]*;" % name, text)
    assert len(arrivals) == 1 and "t == 0" in arrivals[0] and "x == 0" in arrivals[0]  # with tile A's first P alone
    # by the issuer's one warp, or by the four whose rows those are
    assert re.findall(r"mbar_init\(bar\(%s\), (\w+)\)" % name, text) == ["4" if "gt == 0" in arrivals[0] else "1"]
    assert len(re.findall(r"\(bar\(%s\b" % name, text)) == 3  # set up, passed, waited for
