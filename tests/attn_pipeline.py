"""A model of the row-tile attention kernel's roles and barriers, run in random
orders on the CPU.

A block walks pieces (key tiles n, row tiles 1 or 2, a cleared tail or not, the
rows' sums begin, end here).  Its roles are the copy warp, two product warps
and two groups of four softmax warps; copies land in any order, products
complete in the order of their issue.  A barrier is waited on by the parity of
a phase, as in hardware: the wait is met when the phase at hand has the other
parity, also where that is the one two before the phase that was meant.  The
model knows which phase that is and what each buffer holds, and raises Fault
where a wait is met too early, data is not what a role takes it for, or nobody
can move.
"""
import os
import random
import re

from w8a8_int8_quantized_token_gb300 import build_lib

MOST_IDLE = 3000  # rounds in which nothing moved


class Fault(Exception):
    pass


def kernel_counts(D):
    """NS, NB, NO and the arrivals that release the queries, from the kernel."""
    text = open(os.path.join(build_lib.CSRC, "wq_attn_tc.cu")).read()
    pick = lambda name: re.search(r"static constexpr int %s = ([^;]+);" % name, text).group(1)
    ternary = lambda name: [int(x) for x in re.fullmatch(r"D == 128 \? (\d+) : (\d+)", pick(name)).groups()][D != 128]
    return dict(NS=ternary("NS"), NB=ternary("NB"), NO=int(pick("NO")), release=sum(int(x) for x in pick("Q_EMPTY_COUNT").split("+")))


class Barrier:
    def __init__(self, name, count):
        self.name, self.count, self.phase, self.left, self.bytes = name, count, 0, count, 0

    def _turn(self):
        if self.left < 0:
            raise Fault(f"{self.name}: too many arrivals")
        if self.left == 0 and self.bytes == 0:
            self.phase, self.left = self.phase + 1, self.count

    def arrive(self):
        self.left -= 1
        self._turn()

    def expect(self, n):
        self.bytes += n
        self.arrive()

    def landed(self):
        self.bytes -= 1
        self._turn()


def need(cond, what):
    if not cond:
        raise Fault(what)


def run(D, pieces, seed, NS, NB, NO, release, softmax_waits=True, last_two=True):
    """Runs a block over `pieces` = [(n, tiles, tail, open, close)].  With
    `release` 10 the product warps take part in the release of the queries;
    without `softmax_waits` idle softmax warps wait for them only where they
    release them; without `last_two` a piece's end is waited for by its last
    product's signal alone."""
    R = random.Random(seed)
    NSB = 2 * NB if NB % 2 else NB
    full = [Barrier(f"full {i}", 1) for i in range(NS)]
    empty = [Barrier(f"empty {i}", 2) for i in range(NS)]
    q_full, q_empty = Barrier("queries", 1), Barrier("queries released", release)
    scores = [Barrier(f"scores {i}", 1) for i in range(NSB)]
    weights = [[Barrier(f"weights {i} {h}", 4) for h in range(2)] for i in range(NSB)]
    done = [[Barrier(f"products of {t}, {i}", 1) for i in range(NO)] for t in range(2)]
    cleared = [Barrier(f"tail {i}", 1) for i in range(2)]
    bars = full + empty + [q_full, q_empty] + scores + sum(weights, []) + sum(done, []) + cleared
    turn = {1: [0, 0], 2: [0, 0]}  # named barriers of two warps: arrivals, generation
    queue, copies = [], []         # issued products and signals; copies under way
    stage, sbuf, pbuf, acc = [None] * NS, [None] * NB, [[None, None] for _ in range(NB)], [None, None]
    given = {}

    def wait(bar, index):
        """Until phase `index` of the barrier is over, by its parity."""
        while (bar.phase & 1) == (index & 1):
            yield
        need(bar.phase > index, f"{bar.name}: phase {bar.phase} taken for the end of {index}")

    def hand(i):
        turn[i][0] += 1
        if turn[i][0] == 2:
            turn[i] = [0, turn[i][1] + 1]

    def take(i):
        gen = turn[i][1]
        hand(i)
        while turn[i][1] == gen:
            yield

    def copy_warp():
        g = q = tails = 0
        for pi, (n, tiles, tail, opens, _) in enumerate(pieces):
            if opens:
                if q:
                    yield from wait(q_empty, q - 1)
                q_full.expect(tiles)
                copies.extend([(q_full, None, None)] * tiles)
            q += opens
            for j in range(n):
                for kv in "kv":
                    s = g % NS
                    if g >= NS:
                        yield from wait(empty[s], g // NS - 1)
                    full[s].expect(1)
                    copies.append((full[s], s, (pi, j, kv)))
                    g += 1
                    yield
            if tail:
                s = (g - 1) % NS
                yield from wait(full[s], (g - 1) // NS)
                stage[s] = stage[s] + ("cleared",)
                cleared[tails % 2].arrive()
                tails += 1

    def product_warp(t):
        g = kk = q = tails = 0
        ends = [0, 0]
        for pi, (n, tiles, tail, opens, closes) in enumerate(pieces):
            steps, two, each = n * tiles, tiles == 2, NB > tiles
            turns = two and NB == 2
            if turns and t == 1:
                hand(1)
            if opens:
                yield from wait(q_full, q)
                if release > 8:
                    q_empty.arrive()
            q += opens

            def qk(k, pi=pi, g=g, kk=kk, two=two, tiles=tiles):
                j, o = (k >> 1, k & 1) if two else (k, 0)
                s, buf = (g + 2 * j) % NS, (kk + k) % NB

                def product():
                    need(stage[s] == (pi, j, "k"), f"scores of {(pi, j)} read {stage[s]}")
                    sbuf[buf], pbuf[buf] = (pi, j, o), [None, None]
                queue.extend([product, scores[(kk + k) % NSB].arrive])

            def pv(k, h, pi=pi, g=g, kk=kk, two=two, n=n, tail=tail):
                j, o = (k >> 1, k & 1) if two else (k, 0)
                s, buf = (g + 2 * j + 1) % NS, (kk + k) % NB
                want = (pi, j, "v") + (("cleared",) if tail and j == n - 1 else ())

                def product():
                    need(stage[s] == want, f"values {want} read {stage[s]}")
                    need(pbuf[buf][h] == (pi, j, o), f"weights of {(pi, j, o)} are {pbuf[buf][h]}")
                    if h:
                        acc[o] = (pi, j)
                queue.append(product)

            def free(i, tiles=tiles, g=g):
                queue.append(empty[(g + i) % NS].arrive)
                if tiles == 1:
                    empty[(g + i) % NS].arrive()

            first = -NB + ((t - NB) % 2) if two else -NB if t == 0 else steps
            for k in range(first, steps, tiles):
                more = k + NB < steps
                j, jn = (k >> 1, (k + NB) >> 1) if two else (k, k + NB)
                v, c, p = g + 2 * j + 1, g + 2 * jn, kk + k
                if k >= 0:
                    yield from wait(full[v % NS], v // NS)
                    if tail and j + 1 == n:
                        yield from wait(cleared[tails % 2], tails // 2)
                if more:
                    yield from wait(full[c % NS], c // NS)
                if k >= 0:
                    yield from wait(weights[p % NSB][0], p // NSB)
                if turns and (k >= 0 or more):
                    yield from take(1 + t)
                if k >= 0:
                    pv(k, 0)
                    yield from wait(weights[p % NSB][1], p // NSB)
                    pv(k, 1)
                    o = t if two else 0
                    if each or (j + 1 == n and closes):
                        queue.append(done[o][(ends[o] + (j if each else 0)) % NO].arrive)
                if more:
                    qk(k + NB)
                if turns and (k >= 0 or more) and (t == 0 or more):
                    hand(2 - t)
                if k >= 0:
                    free(2 * j + 1)
                if more:
                    free(2 * jn)
                yield
            g, kk, tails = g + 2 * n, kk + steps, tails + tail
            for o in range(tiles):
                ends[o] += n if each else closes

    def softmax_warp(t):
        kk = q = ends = 0
        for pi, (n, tiles, _, opens, closes) in enumerate(pieces):
            each, k, kk = NB > tiles, kk + t, kk + n * tiles
            if opens and (softmax_waits or t >= tiles):
                yield from wait(q_full, q)
            q += opens
            if t >= tiles:
                if closes:
                    q_empty.arrive()
                continue
            for j in range(n):
                yield from wait(scores[k % NSB], k // NSB)
                need(sbuf[k % NB] == (pi, j, t), f"softmax of {(pi, j, t)} reads {sbuf[k % NB]}")
                for _ in range(R.randint(0, 3)):
                    yield
                if (j or not opens) and R.random() < 0.3:  # a maximum grew: the sums are scaled
                    if each:
                        e = ends + j - 1
                        yield from wait(done[t][e % NO], e // NO)
                    before = (pi, j - 1) if j else (pi - 1, pieces[pi - 1][0] - 1)
                    need(acc[t] == before, f"sums of {before} of {t} are {acc[t]}")
                for h in range(2):
                    given[pi, j, t, h] = given.get((pi, j, t, h), 0) + 1
                    if given[pi, j, t, h] == 4:
                        pbuf[k % NB][h] = (pi, j, t)
                    weights[k % NSB][h].arrive()
                    yield
                k += tiles
            if closes:
                e = ends + n - 1 if each else ends
                if each and (n > 1 or not opens) and last_two:
                    yield from wait(done[t][(e - 1) % NO], (e - 1) // NO)
                yield from wait(done[t][e % NO], e // NO)
                need(acc[t] == (pi, n - 1), f"result of {(pi, n - 1, t)} is {acc[t]}")
                for _ in range(R.randint(0, 6)):
                    yield
                q_empty.arrive()
                ends = e + 1
            elif each:
                ends += n

    roles = {"copies": copy_warp(), "products 0": product_warp(0), "products 1": product_warp(1)}
    roles.update({f"softmax {t} {w}": softmax_warp(t) for t in range(2) for w in range(4)})
    slow = {r: R.choice([1, 1, 3, 8]) for r in [*roles, "tensor cores", "memory"]}
    idle, last = 0, None
    while roles:
        for r in R.sample(list(roles), len(roles)):
            if not R.randrange(slow[r]):
                try:
                    next(roles[r])
                except StopIteration:
                    del roles[r]
        if not R.randrange(slow["tensor cores"]):
            for act in queue[:R.randint(1, 3)]:
                queue.pop(0)()
        if copies and not R.randrange(slow["memory"]):
            bar, s, what = copies.pop(R.randrange(min(len(copies), 6)))
            if s is not None:
                stage[s] = what
            bar.landed()
        now = [(b.phase, b.left) for b in bars], len(queue), len(copies), len(roles), str(turn)
        idle, last = (0 if now != last else idle + 1), now
        if idle > MOST_IDLE:
            raise Fault(f"nobody moves: {sorted(roles)}")


def random_pieces(R):
    tail = lambda: R.random() < 0.5
    if R.random() < 0.25:  # prefix and suffix under the same sums
        t = R.choice([1, 2])
        return [(R.randint(1, 7), t, tail(), 1, 0), (R.randint(1, 7), t, tail(), 0, 1)]
    return [(R.randint(1, R.choice([1, 3, 9])), R.choice([1, 2]), tail(), 1, 1) for _ in range(R.randint(1, 6))]
