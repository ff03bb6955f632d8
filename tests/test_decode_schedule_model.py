"""The schedules of the decode kernel and of the many-row kernel, restated in Python and run on random batches (CPU): the
line of work -- for each unit a few places for its start, then one for each key block -- the equal contiguous ranges of
the CTAs, the two slots of each and the parts that the joining kernels add.  Mirrors dec_locate, the loops of
attn_decode_kernel and attn_decode_join_kernel (csrc/attn_decode_kernel.cuh), and rows_locate, the scheduler and
attn_rows_join_kernel (csrc/attn_fwd_rows_kernel.cuh)."""
import random

import pytest


class Line:
    """units: blocks of each unit, in order (0: no place in the line)."""

    def __init__(self, units, over, min_share, ctas):
        self.over, self.ctas = over, ctas
        self.units = units
        self.first, at = [], 0
        for n in units:
            self.first.append(at)
            at += n + over if n else 0
        self.total = at
        self.share = max(min_share, -(-at // ctas))

    def block_at(self, p):
        return max(0, p - self.over)

    def writes(self, cta):
        """(unit, blk0, blk1, whole, slot) of each segment the CTA computes."""
        begin = cta * self.share
        end, out = min(self.total, begin + self.share), []
        for u, n in enumerate(self.units):
            if n == 0:
                continue
            lo, hi = self.first[u], self.first[u] + n + self.over
            x0, x1 = max(lo, begin), min(hi, end)
            if x0 >= x1:
                continue
            b0, b1 = self.block_at(x0 - lo), self.block_at(x1 - lo)
            if b0 < b1:
                out.append((u, b0, b1, b0 == 0 and b1 == n, 2 * cta + (0 if x0 == begin else 1)))
        return out

    def parts(self, u):
        """The slots the joining kernel adds for a unit, or "whole"."""
        u0 = self.first[u]
        u1 = u0 + self.units[u] + self.over
        f, e = (u0 + self.over) // self.share, (u1 - 1) // self.share
        if f == e:
            return "whole"
        return [2 * c + (1 if c == f and u0 > c * self.share else 0) for c in range(f, e + 1)]

    def boundary(self, c):
        """The unit that block c of attn_rows_join_kernel joins, if any."""
        x = (c + 1) * self.share
        if x >= self.total:
            return None
        for u, n in enumerate(self.units):
            if n and self.first[u] <= x < self.first[u] + n + self.over:
                u0 = self.first[u]
                if u0 + self.over < x and (u0 + self.over) // self.share == c:
                    return u, (u0 + n + self.over - 1) // self.share - c + 1, 2 * c + (1 if u0 > c * self.share else 0)
        return None


@pytest.mark.parametrize("form", ["decode", "rows"])
@pytest.mark.parametrize("seed", range(80))
def test_every_block_once_and_every_part_joined(form, seed):
    r = random.Random(seed)
    block, over, least = (64, 2, 4) if form == "decode" else (128, 1, 3)
    lens = [r.choice([0, 1, 63, 64, 65, 128, 129, r.randrange(3000)]) for _ in range(r.choice([1, 2, 3, 7, 40]))]
    heads = r.choice([1, 2, 5])
    units = [max(1, -(-n // block)) if form == "decode" else -(-n // block) for n in lens for _ in range(heads)]
    if form == "decode" and r.random() < 0.2:
        units = [1] * len(units)
        least = 3   # units that are not split
    ln = Line(units, over, least, r.choice([1, 2, 5, 17, 100, 444]))
    whole_only = least == 3 and form == "decode"
    seen, slots, wholes = set(), {}, set()
    for c in range(ln.ctas):
        for u, b0, b1, whole, slot in ln.writes(c):
            for b in range(b0, b1):
                assert (u, b) not in seen
                seen.add((u, b))
            if whole:
                wholes.add(u)
            else:
                assert not whole_only and slot not in slots and slot < 2 * ln.ctas
                slots[slot] = (u, b0, b1)
    assert len(seen) == sum(units)
    if form == "rows":   # the joining kernel goes by the CTAs' boundaries: each split unit once, with these parts
        joined = [b for b in map(ln.boundary, range(ln.ctas - 1)) if b]
        assert sorted(u for u, _, _ in joined) == sorted(u for u, n in enumerate(units) if n and ln.parts(u) != "whole")
        for u, n, first in joined:
            assert ln.parts(u) == [first] + [2 * (first // 2 + k) for k in range(1, n)]
    for u, n in enumerate(units):
        if n == 0:
            continue
        got = ln.parts(u)
        if got == "whole":
            assert u in wholes
            continue
        at = 0
        for s in got:   # in key order, without a gap
            unit, b0, b1 = slots.pop(s)
            assert unit == u and b0 == at
            at = b1
        assert at == n
    assert not slots   # nothing computed that no one reads
