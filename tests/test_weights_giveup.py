"""The attention-weights kernel after a wait that ran out, in a model of its
roles: whichever role gives up, at whichever wait, every role ends.

Waits on memory barriers end by themselves (their limit, or the flag that
another role's limit sets); the barrier at which the four warps of a key tile
exchange log-sum-exps has no limit, so none of the four may be left there."""
import random

import pytest
from test_weights_pipeline import Kernel, work

BATCH = 4


class Meeting:
    """A barrier of four warps without a limit; all of them get the AND of what they bring."""

    def __init__(self):
        self.brought, self.got, self.round = [], {}, 0

    def come(self, ok):
        self.brought.append(ok)
        mine = self.round
        if len(self.brought) == 4:
            self.got[mine], self.brought, self.round = all(self.brought), [], mine + 1
        return mine


class GivingUp(Kernel):
    def __init__(self, *args, together=True, batch=BATCH):
        super().__init__(*args)
        self.together, self.batch = together, batch
        self.meet, self.abort = [Meeting(), Meeting()], False
        self.read = [[0, 0], [0, 0]]

    def warp(self, g):
        """A weighing warp.  What it yields is (condition, whether the wait has a limit); it is sent whether it passed."""
        st, ok = 0, True
        for n, piece in enumerate(self.pieces):
            for k in range(piece[0]):
                for q in range(piece[2], piece[3]):
                    if k == 0 and (q - piece[2]) % self.batch == 0:
                        mine = self.meet[g].come(ok)
                        yield lambda: mine in self.meet[g].got, False
                        if self.together and not self.meet[g].got[mine]:
                            return
                    if g >= self.tiles(piece, k) or not ok:
                        continue
                    buf = st & 1
                    ok = yield lambda: self.sf[g][buf].passed((st >> 1) & 1), True
                    if not ok:
                        self.abort = True
                        if not self.together:
                            return
                        continue
                    assert self.s[g][buf] == (n, k, g, q)
                    self.read[g][buf] += 1
                    if self.read[g][buf] == 4:
                        self.s[g][buf], self.read[g][buf] = None, 0
                    self.se[g][buf].arrive()
                    st += 1

    def run(self, who, when):
        """Role `who` gives up at its wait number `when`, if it has so many; the others once they find the flag."""
        def with_limits(role):
            for cond in role:
                if not (yield cond, True):
                    self.abort = True
                    return

        roles = [with_limits(r) for r in (self.producer(), self.mma(0), self.mma(1))]
        roles += [self.warp(g) for g in (0, 1) for _ in range(4)]
        waits, count = [next(r, None) for r in roles], [0] * len(roles)
        bias = [self.r.choice([1, 1, 5, 30]) for _ in range(len(roles) + 4)]
        gave = False
        while any(w is not None for w in waits) or self.flying or any(self.queue):
            can = [("pass", i) for i, w in enumerate(waits) if w is not None and w[0]()]
            can += [("fail", i) for i, w in enumerate(waits) if w is not None and w[1] and not w[0]() and self.abort]
            if not gave and waits[who] is not None and waits[who][1] and count[who] >= when and not waits[who][0]():
                can.append(("fail", who))
            can += [("land", i) for i in range(len(self.flying))] + [("job", g) for g in range(2) if self.queue[g]]
            if not can:
                return [i for i, w in enumerate(waits) if w is not None]
            kind, i = self.r.choices(can, [bias[j if kind in ("pass", "fail") else len(roles) + j % 4] for kind, j in can])[0]
            if kind == "land":
                to, slot, what, bar = self.flying.pop(i)
                to[slot] = what
                bar.land(1)
            elif kind == "job":
                self.step(i)
            else:
                count[i] += 1
                gave |= kind == "fail"
                try:
                    waits[i] = roles[i].send(kind == "pass")
                except StopIteration:
                    waits[i] = None
        return []


def left(seed, **kw):
    r = random.Random(seed)
    k = GivingUp(work(r) + work(r), r.choice([2, 3, 4, 6, 8]), r.choice([2, 3, 4, 8]), r, batch=r.choice([1, BATCH]), **kw)
    return k.run(r.randrange(11), r.randint(0, 12))


@pytest.mark.parametrize("seed", range(400))
def test_every_role_ends_whoever_gives_up(seed):
    assert left(seed) == []


def test_the_model_finds_warps_that_leave_by_themselves():
    """Each warp leaving as soon as its own wait fails, as the kernel must not:
    some order leaves others of its key tile at their barrier."""
    stuck = [left(seed, together=False) for seed in range(400)]
    assert any(stuck) and all(i >= 3 for s in stuck for i in s)
