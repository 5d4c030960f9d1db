"""A randomized CPU model of the 4-bit GEMM of few tokens: the CTAs of a cluster with their
producer warp, issuing warp and four more, which code the tokens into the stages (if the kernel
quantizes) and then take the accumulator, and the join of the CTAs' partial tiles.

A stage's `full` barrier takes the producer's arrival with the bytes of its loads, and with
quantization one arrival of each coding warp; `empty` the commit of its products.  The partial
tile lies where the stages were: no load may be in flight there and no product unfinished when
a warp writes it.  All CTAs' tiles are written before one is read (first cluster barrier), and no
CTA leaves before all have read (second).

Loads land at any time, products run in order after their issue, a commit arrives when they are
done.  Leaving out any of the waits must be caught."""
import random

import pytest


class MBarrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = self.phases = 0

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.phases += 1
            self.pending = self.count

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        assert self.pending >= 0, "arrival beyond the barrier's count"
        self._check()

    def complete(self):
        self.tx -= 1
        self._check()

    def passed(self, parity):
        return (self.phases & 1) != parity


class Meeting:
    """A barrier that everybody waits at."""

    def __init__(self, n):
        self.n, self.here, self.turn = n, 0, 0

    def wait(self, skip=False):
        mine = self.turn
        self.here += 1
        if self.here == self.n:
            self.here, self.turn = 0, self.turn + 1
        while self.turn == mine and not skip:
            yield


def run(splits, slices, stages, quant, seed, drop=""):
    rng = random.Random(seed)
    cluster = [Meeting(6 * splits), Meeting(6 * splits)]
    ctas, actors, pipes, landing = [], [], [], []

    class Cta:
        pass

    for r in range(splits):
        c = Cta()
        c.range = range(slices * r // splits, slices * (r + 1) // splits)
        c.full = [MBarrier(5 if quant else 1) for _ in range(stages)]
        c.empty = [MBarrier(1) for _ in range(stages)]
        c.tfull = MBarrier(1)
        c.stage = [{} for _ in range(stages)]
        c.queue, c.done, c.sum = [], 0, 0
        c.block = Meeting(6)
        c.part, c.left = set(), 0
        c.coded = Meeting(4)
        ctas.append(c)

    pieces = ("w", "sw") if quant else ("w", "sw", "x", "sx")

    def producer(r):
        c = ctas[r]
        for it, ks in enumerate(c.range):
            s, ph = it % stages, (it // stages) & 1
            while drop != "empty" and not c.empty[s].passed(ph ^ 1):
                yield
            c.full[s].arrive(tx=len(pieces))
            for p in pieces:
                landing.append((r, s, p, ks))
            yield
        yield from end(r, None)

    def issuer(r):
        c = ctas[r]
        for it, ks in enumerate(c.range):
            s, ph = it % stages, (it // stages) & 1
            while drop != "full" and not c.full[s].passed(ph):
                yield
            c.queue.append(("mma", s, ks))
            c.queue.append(("commit", c.empty[s]))
            if ks == c.range[-1]:
                c.queue.append(("commit", c.tfull))
            yield
        yield from end(r, None)

    def tensor(c):
        while True:
            if c.queue:
                op = c.queue[0]
                if op[0] == "mma":
                    for k in range(4):
                        want = set(pieces) | ({f"x{w}" for w in range(4)} if quant else set())
                        assert all(c.stage[op[1]].get(p) == op[2] for p in want), "product of another slice"
                        if k < 3:
                            yield
                    c.sum += 1
                    c.done += 1
                else:
                    op[1].arrive()
                c.queue.pop(0)
            yield

    def worker(r, w):
        c = ctas[r]
        if quant:
            for it, ks in enumerate(c.range):
                s, ph = it % stages, (it // stages) & 1
                while drop != "coder" and not c.empty[s].passed(ph ^ 1):
                    yield
                c.stage[s][f"x{w}"] = ks
                yield
                c.full[s].arrive()
                yield
            yield from c.coded.wait()
        while drop != "tfull" and not c.tfull.passed(0):
            yield
        assert c.done == len(c.range), "the accumulator read before it is complete"
        assert not any(q[0] == r for q in landing), "the partial tile written over a load in flight"
        c.part.add(w)
        yield
        yield from end(r, w)

    def end(r, w):
        c = ctas[r]
        yield from c.block.wait()
        if splits == 1:
            return
        yield from cluster[0].wait(skip=drop == "first")
        if w is not None:
            for q in range(splits):
                assert ctas[q].left < 6, "a CTA has left whose tile is still read"
                assert len(ctas[q].part) == 4, "a partial tile read before it is written"
                yield
        yield from cluster[1].wait(skip=drop == "second")
        c.left += 1

    for r in range(splits):
        actors += [producer(r), issuer(r)] + [worker(r, w) for w in range(4)]
        pipes.append(tensor(ctas[r]))
    weights = [rng.choice((1, 1, 3, 20)) for _ in actors]
    alive = list(range(len(actors)))
    for _ in range(200000):
        if not alive:
            return
        x = rng.random()
        if x < 0.25:
            next(rng.choice(pipes))
        elif x < 0.5 and landing:
            r, s, p, ks = landing.pop(rng.randrange(len(landing)))
            ctas[r].stage[s][p] = ks
            ctas[r].full[s].complete()
        else:
            a = rng.choices(alive, [weights[k] for k in alive])[0]
            try:
                next(actors[a])
            except StopIteration:
                alive.remove(a)
    raise AssertionError("no progress")


@pytest.mark.parametrize("quant", [False, True])
@pytest.mark.parametrize("splits,slices,stages", [(1, 1, 4), (1, 9, 3), (2, 8, 4), (4, 18, 4), (8, 67, 3)])
def test_every_schedule_is_ordered(splits, slices, stages, quant):
    for seed in range(12):
        run(splits, slices, stages, quant, seed)


@pytest.mark.parametrize("quant,drop", [(False, d) for d in ("empty", "full", "tfull", "first", "second")]
                         + [(True, d) for d in ("empty", "coder", "full", "tfull", "first", "second")])
def test_a_missing_wait_is_caught(quant, drop):
    caught = 0
    for seed in range(30):
        try:
            run(2, 14, 3, quant, seed, drop)
        except AssertionError:
            caught += 1
    assert caught >= 8, f"{drop}: {caught}"
