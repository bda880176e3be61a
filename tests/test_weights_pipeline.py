"""A model of the attention-weights kernel's roles and barriers, run in random
orders on the CPU: no slot is read before it is full or filled while it is read,
no barrier gets an arrival too many, and every role ends."""
import random

import pytest


class Barrier:
    def __init__(self, count):
        self.count, self.left, self.tx, self.phase = count, count, 0, 0

    def arrive(self, tx=0):
        assert self.left > 0, "an arrival too many"
        self.left -= 1
        self.tx += tx
        self.turn()

    def land(self, tx):
        self.tx -= tx
        self.turn()

    def turn(self):
        if self.left == 0 and self.tx == 0:
            self.phase += 1
            self.left = self.count

    def passed(self, parity):
        return (self.phase & 1) != parity


class Kernel:
    """pieces: (pairs, tiles of the last pair, first query tile, end) of one block."""

    def __init__(self, pieces, nk, nq, r, observe=True):
        self.pieces, self.nk, self.nq, self.r, self.observe = pieces, nk, nq, r, observe
        both = 2 if observe else 1
        self.kf, self.ke = [Barrier(1) for _ in range(nk)], [Barrier(both) for _ in range(nk)]
        self.qf, self.qe = [Barrier(1) for _ in range(nq)], [Barrier(2) for _ in range(nq)]
        self.sf = [[Barrier(1), Barrier(1)] for _ in range(2)]
        self.se = [[Barrier(4), Barrier(4)] for _ in range(2)]
        self.k, self.q = [None] * nk, [None] * nq          # what a slot holds
        self.s = [[None, None], [None, None]]
        self.flying, self.queue, self.seen = [], [[], []], [[], []]

    def tiles(self, piece, k):
        return piece[1] if k + 1 == piece[0] else 2

    def producer(self):
        ks, kp, qs, qp = 0, 1, 0, 1
        for n, piece in enumerate(self.pieces):
            for k in range(piece[0]):
                if piece[2] == piece[3]:
                    continue
                for g in range(self.tiles(piece, k)):
                    yield lambda: self.ke[ks].passed(kp)
                    self.kf[ks].arrive(1)
                    self.k[ks] = None
                    self.flying.append((self.k, ks, (n, k, g), self.kf[ks]))
                    ks, kp = (ks + 1, kp) if ks + 1 < self.nk else (0, kp ^ 1)
                for q in range(piece[2], piece[3] if k == 0 else piece[2]):
                    yield lambda: self.qe[qs].passed(qp)
                    self.qf[qs].arrive(1)
                    self.q[qs] = None
                    self.flying.append((self.q, qs, (n, q), self.qf[qs]))
                    qs, qp = (qs + 1, qp) if qs + 1 < self.nq else (0, qp ^ 1)

    def mma(self, g):
        ks, kp, qs, qp, st = 0, 0, 0, 0, 0
        for n, piece in enumerate(self.pieces):
            if piece[2] == piece[3]:
                continue
            for k in range(piece[0]):
                two = self.tiles(piece, k) == 2
                tile = g == 0 or two
                k1, kp1 = (ks + 1, kp) if ks + 1 < self.nk else (0, kp ^ 1)
                kg, other = (k1, ks) if g else (ks, k1)
                if self.observe:
                    yield lambda: self.kf[ks].passed(kp)
                    if two:
                        yield lambda: self.kf[k1].passed(kp1)
                    if g or two:
                        self.ke[other].arrive()
                elif tile:
                    yield lambda: self.kf[kg].passed(kp1 if g else kp)
                for q in range(piece[2], piece[3]):
                    done = k + 1 == piece[0]
                    if k == 0:
                        yield lambda: self.qf[qs].passed(qp)
                    if tile:
                        buf = st & 1
                        yield lambda: self.se[g][buf].passed(((st >> 1) & 1) ^ 1)
                        job = [("mma", kg, (n, k, g), qs, (n, q), buf)]
                        if q + 1 == piece[3]:
                            job.append(("arrive", self.ke[kg]))
                        if done:
                            job.append(("arrive", self.qe[qs]))
                        job.append(("arrive", self.sf[g][buf]))
                        self.queue[g] += job
                        st += 1
                    elif done:
                        self.queue[g].append(("arrive", self.qe[qs]))
                    if done:
                        qs, qp = (qs + 1, qp) if qs + 1 < self.nq else (0, qp ^ 1)
                ks, kp = (k1, kp1) if two else (ks, kp)
                ks, kp = (ks + 1, kp) if ks + 1 < self.nk else (0, kp ^ 1)

    def weights(self, g):
        st = 0
        for n, piece in enumerate(self.pieces):
            for k in range(piece[0]):
                for q in range(piece[2], piece[3]):
                    if g >= self.tiles(piece, k):
                        continue
                    buf = st & 1
                    yield lambda: self.sf[g][buf].passed((st >> 1) & 1)
                    assert self.s[g][buf] == (n, k, g, q)
                    self.seen[g].append(self.s[g][buf])
                    self.s[g][buf] = None
                    for _ in range(4):
                        self.se[g][buf].arrive()
                    st += 1

    def step(self, g):
        job = self.queue[g].pop(0)
        if job[0] == "arrive":
            return job[1].arrive()
        _, ks, key, qs, query, buf = job
        assert self.k[ks] == key and self.q[qs] == query, "a product reads a slot that is not its own"
        assert self.s[g][buf] is None, "scores that nobody has read are written over"
        self.s[g][buf] = (*key, query[1])

    def run(self):
        roles = [self.producer(), self.mma(0), self.mma(1), self.weights(0), self.weights(1)]
        waits = [(lambda: True)] * len(roles)
        bias = [self.r.choice([1, 1, 5, 30]) for _ in range(9)]  # some parts are slow
        while any(w is not None for w in waits) or self.flying or any(self.queue):
            can = [("role", i) for i, w in enumerate(waits) if w is not None and w()]
            can += [("land", i) for i in range(len(self.flying))] + [("job", g) for g in range(2) if self.queue[g]]
            assert can, "all roles wait"
            kind, i = self.r.choices(can, [bias[(j if kind == "role" else 5 + j % 4)] for kind, j in can])[0]
            if kind == "land":
                to, slot, what, bar = self.flying.pop(i)
                to[slot] = what
                bar.land(1)
            elif kind == "job":
                self.step(i)
            else:
                waits[i] = next(roles[i], None)
        for g in range(2):
            assert self.seen[g] == [(n, k, g, q) for n, p in enumerate(self.pieces) for k in range(p[0])
                                    for q in range(p[2], p[3]) if g < self.tiles(p, k)]


def work(r):
    pieces = []
    for _ in range(r.randint(1, 6)):
        if r.random() < 0.5:  # one query tile, a run of pairs
            pieces.append((r.randint(1, 6), r.randint(1, 2), 0, r.choice([0, 1, 1, 1])))
        else:
            qa = r.randint(0, 5)
            pieces.append((1, r.randint(1, 2), qa, qa + r.randint(1, 7)))
    return pieces


@pytest.mark.parametrize("seed", range(300))
def test_any_order_of_the_roles(seed):
    r = random.Random(seed)
    Kernel(work(r), r.choice([2, 3, 4, 6, 8]), r.choice([2, 3, 4, 8]), r).run()


def test_the_model_finds_a_slot_that_one_warp_passes_over():
    """Each product warp waiting for its own key tile alone, as the kernel must
    not: some order reads a slot too early, or gives a barrier one arrival more
    than it takes."""
    failed = 0
    for seed in range(300):
        r = random.Random(seed)
        try:
            Kernel(work(r), r.choice([3, 4, 6]), 2, r, observe=False).run()
        except AssertionError:
            failed += 1
    assert failed
