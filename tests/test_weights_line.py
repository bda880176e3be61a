"""A model of how the attention-weights kernel's blocks share its line of units
(sequence, key head, pair of key tiles, query tile), on the CPU: every unit that
has work is taken once, and the join adds every part of a cut pair once."""
import random

import pytest

PAIR = 256


class Seq:
    def __init__(self, n, length, tpt):
        self.n, self.len, self.tpt = n, length, tpt
        self.shift = tpt.bit_length() - 1
        self.old = length - n
        self.pairs = -(-length // PAIR)
        self.tiles = -(-n // tpt)
        self.costs = -(-n // (1 << self.shift))
        self.p1 = 0 if self.old <= 0 else -(-self.old // PAIR)
        self.d1 = self.p1 * PAIR - self.old

    def cost(self, p):
        return 1 if self.tiles <= 1 else self.costs - max(0, (p * PAIR - self.old) >> self.shift)

    def before(self, p):
        if self.tiles <= 1:
            return p
        m = max(0, p - self.p1)
        return p * self.costs - (m * (self.d1 >> self.shift) + (PAIR >> self.shift) * (m * (m - 1) // 2))


def place(seqs, heads, at):
    for b, s in enumerate(seqs):
        c = s.before(s.pairs) * heads
        if at < c:
            return b, at
        at -= c


def begin(seqs, heads, at):
    b, off = place(seqs, heads, at)
    s = seqs[b]
    h, rest = divmod(off, s.before(s.pairs))
    lo, hi = 0, s.pairs - 1
    while lo < hi:
        mid = (lo + hi + 1) // 2
        lo, hi = (mid, hi) if s.before(mid) <= rest else (lo, mid - 1)
    return b, h, lo, rest - s.before(lo)


def pieces(seqs, heads, at, left):
    if left <= 0:
        return
    b, h, p, u = begin(seqs, heads, at)
    while left > 0:
        while p >= seqs[b].pairs:
            p = 0
            if seqs[b].pairs > 0:
                h += 1
                if h < heads:
                    break
            h, b = 0, b + 1
        s = seqs[b]
        if s.tiles <= 1:
            take = min(s.pairs - p, left)
            for k in range(take):
                yield b, h, p + k, 0, s.tiles, True, 0
            left -= take
            p += take
            continue
        first, cost = max(0, (p * PAIR - s.old) // s.tpt), s.cost(p)
        tiles, take = s.tiles - first, min(cost - u, left)
        assert cost >= 1 and tiles >= 1
        yield b, h, p, first + u * tiles // cost, first + (u + take) * tiles // cost, take == cost, 1 if u == 0 else 0
        left -= take
        u += take
        if u == cost:
            u, p = 0, p + 1


@pytest.mark.parametrize("seed", range(200))
def test_every_unit_is_taken_once_and_every_part_joined(seed):
    r = random.Random(seed)
    tpt, heads = r.choice([1, 2, 3, 16, 18, 25, 42, 64, 100, 128]), r.randint(1, 4)
    most = r.choice([1, 3, 40, 700, 3000])
    seqs = []
    for _ in range(r.randint(1, 9)):
        n = r.choice([0, 1, r.randint(1, most)])
        seqs.append(Seq(n, r.choice([0, n, max(0, n - r.randint(0, 9)), n + r.randint(0, 2000)]), tpt))
    total = sum(s.before(s.pairs) * heads for s in seqs)
    blocks = r.choice([1, 2, 7, 152])
    cut = [total * c // blocks for c in range(blocks + 1)]
    taken, parts = {}, {}
    for c in range(blocks):
        for b, h, p, qa, qb, whole, slot in pieces(seqs, heads, cut[c], cut[c + 1] - cut[c]):
            for q in range(qa, qb):
                assert (b, h, p, q) not in taken
                taken[b, h, p, q] = (c, slot)
            if not whole:
                assert (c, slot) not in parts
                parts[c, slot] = (b, h, p)
    want = {(b, h, p, q) for b, s in enumerate(seqs) for h in range(heads) for p in range(s.pairs)
            for q in range(s.tiles) if s.tiles == 1 or p * PAIR <= s.old + min(s.n, (q + 1) * s.tpt) - 1}
    assert set(taken) == want
    joined = set()
    for c in range(blocks - 1):
        at = cut[c + 1]
        if at >= total:
            continue
        b, h, p, u = begin(seqs, heads, at)
        start = at - u
        if u == 0 or start < cut[c]:
            continue
        end = start + seqs[b].cost(p)
        assert seqs[b].cost(p) == seqs[b].before(p + 1) - seqs[b].before(p)
        # a block without units, where there are fewer than blocks, leaves no part
        for k in [(c, 1)] + [(k, 0) for k in range(c + 1, blocks) if cut[k] < min(end, cut[k + 1])]:
            assert parts[k] == (b, h, p) and k not in joined
            joined.add(k)
    assert joined == set(parts)
