"""The decode kernel's schedule, restated in Python and run on random batches (CPU): the line of 64-key blocks, the
equal contiguous ranges of the CTAs, the two slots of each and the parts that the joining kernel adds.  Mirrors
dec_locate and the loops of attn_decode_kernel / attn_decode_join_kernel (csrc/attn_decode_kernel.cuh)."""
import random

import pytest

BLOCK = 64


def blocks_of(n):
    return max(1, -(-n // BLOCK))


class Line:
    def __init__(self, lens, hkv, row_blocks, prefix_len, prefix_row_blocks, min_share, ctas):
        self.lens, self.hkv, self.rb = lens, hkv, row_blocks
        self.pre_nblk = blocks_of(prefix_len) if prefix_len else 0
        self.pre_rb, self.prefix_len = prefix_row_blocks, prefix_len
        self.prefix = hkv * prefix_row_blocks * self.pre_nblk
        self.first = []
        at = self.prefix
        for n in lens:
            self.first.append(at)
            at += hkv * row_blocks * blocks_of(n)
        self.total = at
        self.share = max(min_share, -(-at // ctas))

    def locate(self, x):
        if x < self.prefix:
            return -1, 0
        for b, n in enumerate(self.lens):
            if x < self.first[b] + self.hkv * self.rb * blocks_of(n):
                return b, self.first[b]
        return len(self.lens), 0


def cta_writes(ln, cta):
    """(unit key, blk0, blk1, whole, slot) of each segment the CTA computes."""
    begin, out = cta * ln.share, []
    end = min(ln.total, begin + ln.share)
    seq, first = ln.locate(begin)
    x = begin
    while x < end:
        nblk = ln.pre_nblk if seq < 0 else blocks_of(ln.lens[seq])
        rbs = ln.pre_rb if seq < 0 else ln.rb
        unit, blk0 = divmod(x - first, nblk)
        blk1 = min(nblk, blk0 + end - x)
        h, rb = divmod(unit, rbs)
        out.append(((seq, h, rb), blk0, blk1, blk0 == 0 and blk1 == nblk, 2 * cta + (0 if x == begin else 1)))
        x += blk1 - blk0
        n = ln.hkv * rbs * nblk
        if x >= first + n:
            first += n
            seq += 1
    return out


def parts(ln, u0, u1):
    """The slots the joining kernel adds for a unit, or "whole"."""
    c0, c1 = u0 // ln.share, (u1 - 1) // ln.share
    if c0 == c1:
        return "whole"
    return [2 * c + (1 if c == c0 and u0 != c * ln.share else 0) for c in range(c0, c1 + 1)]


@pytest.mark.parametrize("seed", range(60))
def test_every_block_once_and_every_part_joined(seed):
    r = random.Random(seed)
    B, hkv, rb = r.choice([1, 2, 3, 7, 40]), r.choice([1, 2, 5]), r.choice([1, 1, 3])
    lens = [r.choice([0, 1, 63, 64, 65, r.randrange(3000)]) for _ in range(B)]
    prefix = r.choice([0, 0, 1, 64, 1000])
    min_share = 2
    ctas = r.choice([1, 2, 5, 17, 100, 444])
    ln = Line(lens, hkv, rb, prefix, r.choice([1, 2]) if prefix else 0, min_share, ctas)
    seen, slots, wholes = {}, {}, set()
    for c in range(ctas):
        for key, b0, b1, is_whole, slot in cta_writes(ln, c):
            for blk in range(b0, b1):
                assert (key, blk) not in seen
                seen[key, blk] = c
            if is_whole:
                wholes.add(key)
            else:
                assert slot not in slots and slot < 2 * ctas
                slots[slot] = (key, b0, b1)
    assert len(seen) == ln.total
    units = [(-1, h, q) for h in range(hkv) for q in range(ln.pre_rb if prefix else 0)]
    units += [(b, h, q) for b in range(B) for h in range(hkv) for q in range(rb)]
    for seq, h, q in units:
        nblk = ln.pre_nblk if seq < 0 else blocks_of(lens[seq])
        u0 = (0 if seq < 0 else ln.first[seq]) + (h * (ln.pre_rb if seq < 0 else rb) + q) * nblk
        got = parts(ln, u0, u0 + nblk)
        if got == "whole":
            assert (seq, h, q) in wholes
            continue
        at = 0
        for s in got:   # in key order, without a gap
            key, b0, b1 = slots.pop(s)
            assert key == (seq, h, q) and b0 == at
            at = b1
        assert at == nblk
    assert not slots   # nothing computed that no one reads
