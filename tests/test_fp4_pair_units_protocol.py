"""A randomized CPU model of the 4-bit GEMM's pair kernel with whole and half units, tensor
memory by columns and every wait of the kernel: the producers' of both CTAs, the issuing
thread's four, the epilogue warps'.

Two accumulators of 256 columns overlap by 96 (nvfp4) or 48 (mxfp4), in cells of 16 columns here.
A half unit, a tile cut along N, multiplies and stores 128 columns from its accumulator's first
on, and its slices are four loads a CTA instead of six.  Epilogues as in the kernel: with TMA
stores four warps a CTA read two steps of 64 columns at once, from the end that the accumulators
share, and then say that the shared columns are free, and after two more (a half unit: at once)
that the accumulator is; otherwise eight warps, each with half of the columns, go in steps of 32.

What the hardware orders is all that the model orders: products run in issue order, a scale copy
before the products issued after it but possibly ahead of earlier ones, a commit arrives when
everything issued before it is done, loads land at any time.  Under random schedules, some with
slow warps, a product must find its own slice whole and its scales, must write no columns that a
warp has still to read, and a warp must find its own unit.

Leaving out any of the waits must be caught in a good part of the schedules.  The one exception
is the issuing thread's wait for the accumulator with TMA stores: every warp says that the last
unit's shared columns are free after it has read the unit before whole, so that wait is implied
there, and leaving it out must change nothing."""
import random

import pytest

STAGES = 5
CELL = 16


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


def run(units, slices, tma, overlap, seed, drop="", slow=()):
    """units: a text of W (whole) and H (half); overlap: columns that the accumulators share."""
    rng = random.Random(seed)
    warps = 4 if tma else 8
    full = [MBarrier(1) for _ in range(STAGES)]                       # the even CTA's
    empty = [[MBarrier(1) for _ in range(STAGES)] for _ in range(2)]
    tfull = [[MBarrier(1), MBarrier(1)] for _ in range(2)]
    tshared = MBarrier(8)
    tdrained = [MBarrier(2 * warps), MBarrier(2 * warps)]
    base = (0, 256 - overlap)
    slots = [[{} for _ in range(STAGES)] for _ in range(2)]           # piece -> slice
    scales = [None, None]
    owner, unread = {}, {}                                            # by cell of tensor memory
    landing, queue, cps = [], [], []
    done = {"mma": -1}

    def pieces(i):
        return ("a", "b", "sa", "sb") + (("b2", "sb2") if units[i] == "W" else ())

    def cells(i):
        first = base[i & 1]
        return range(first // CELL, (first + (256 if units[i] == "W" else 128)) // CELL)

    def steps(i, w):
        """The groups of cells that warp w reads of unit i, in order, up to where it says that
        the shared columns are free and up to the end."""
        buf, first = i & 1, base[i & 1]
        if tma:
            n = 4 if units[i] == "W" else 2
            order = [n - 1 - k if buf == 0 else k for k in range(n)]
            cols = [range(first + 64 * k, first + 64 * k + 64, CELL) for k in order]
            return [sum(([c // CELL for c in g] for g in cols[:2]), []), sum(([c // CELL for c in g] for g in cols[2:]), [])]
        part = w // 4
        order = [3 - k if buf == 0 else k for k in range(4)]
        cols = [[c // CELL for c in range(first + part * 128 + 32 * k, first + part * 128 + 32 * k + 32, CELL)] for k in order]
        return [sum(cols[:3], []), cols[3]]

    def holds_shared(i, w):
        return tma or w // 4 != (i & 1)

    def producer(cta):
        it = 0
        for i in range(len(units)):
            for _ in range(slices):
                s, ph = it % STAGES, (it // STAGES) & 1
                while drop != "empty" and not empty[cta][s].passed(ph ^ 1):
                    yield
                if cta == 0:
                    full[s].arrive(tx=2 * len(pieces(i)))
                for p in pieces(i):
                    landing.append((cta, s, p, it))
                it += 1
                yield

    def issuer():
        it = 0
        for i in range(len(units)):
            while i > 1 and drop != "drained" and not tdrained[i & 1].passed(((i >> 1) - 1) & 1):
                yield
            while i > 0 and drop != "shared" and not tshared.passed((i - 1) & 1):
                yield
            for ks in range(slices):
                s, ph = it % STAGES, (it // STAGES) & 1
                while it >= 2 and drop != "scales" and not empty[0][(it - 2) % STAGES].passed(((it - 2) // STAGES) & 1):
                    yield
                while drop != "full" and not full[s].passed(ph):
                    yield
                cps.append((it, i))
                queue.append(("mma", it, i, ks))
                queue.append(("commit", [empty[0][s], empty[1][s]]))
                if ks == slices - 1:
                    queue.append(("commit", [tfull[0][i & 1], tfull[1][i & 1]]))
                it += 1
                yield

    def whole(it, i):
        return all(slots[c][it % STAGES].get(p) == it for c in range(2) for p in pieces(i))

    def copy_scales():
        it, i = cps.pop(0)
        assert done["mma"] >= it - 2, "scales replaced before the products that use them"
        assert whole(it, i), "scales of another slice copied"
        scales[it & 1] = it

    def tensor():
        while True:
            if queue and queue[0][0] == "commit":
                for bar in queue.pop(0)[1]:
                    bar.arrive()
            elif queue:
                _, it, i, ks = queue[0]
                while cps and cps[0][0] <= it:
                    copy_scales()
                if ks == 0:
                    for c in cells(i):
                        assert not unread.get(c), "columns written before they were read"
                        owner[c] = i
                for k in range(4):
                    assert whole(it, i), "product of another slice"
                    assert scales[it & 1] == it, "product with another slice's scales"
                    if k < 3:
                        yield
                if ks == slices - 1:
                    for c in cells(i):
                        assert owner[c] == i
                        unread[c] = {(cta, w) for cta in range(2) for w in range(warps) if any(c in g for g in steps(i, w))}
                done["mma"] = it
                queue.pop(0)
            yield

    def epilogue(cta, w):
        for i in range(len(units)):
            buf = i & 1
            while drop != "tfull" and not tfull[cta][buf].passed((i >> 1) & 1):
                yield
            for k, group in enumerate(steps(i, w)):
                for c in group:
                    if c in cells(i):       # a half unit's other columns are read by no one
                        assert owner.get(c) == i and (cta, w) in unread.get(c, ()), "accumulator of another unit"
                        unread[c].discard((cta, w))
                if group and not tma:
                    yield
                if k == 0 and holds_shared(i, w):
                    tshared.arrive()
                if k == 1:
                    tdrained[buf].arrive()
                yield

    actors = [producer(0), producer(1), issuer()] + [epilogue(c, w) for c in range(2) for w in range(warps)]
    weights = [rng.choice((1, 1, 3, 10)) for _ in actors]
    for w in slow:
        weights[3 + w] *= 0.02
    pipe = tensor()
    speed = rng.choice((0.05, 0.15, 0.3))
    alive = list(range(len(actors)))
    for _ in range(300000):
        if not alive:
            assert not any(unread.values()), "columns never read"
            return
        x = rng.random()
        if x < speed:
            next(pipe)
        elif x < 0.55 and landing:
            cta, s, p, it = landing.pop(rng.randrange(len(landing)))
            slots[cta][s][p] = it
            full[s].complete()
        elif x < 0.6 and cps:
            copy_scales()
        else:
            a = rng.choices(alive, [weights[k] for k in alive])[0]
            try:
                next(actors[a])
            except StopIteration:
                alive.remove(a)
    raise AssertionError("no progress")


# Half units are the last ones of a pair; without TMA stores there are none.
@pytest.mark.parametrize("overlap", [96, 48])
@pytest.mark.parametrize("units,slices,tma", [("W", 1, True), ("H", 1, True), ("WW", 1, True), ("WWWWW", 1, True), ("WWWH", 3, True),
                                              ("WWH", 7, True), ("WHH", 2, True), ("HH", 12, True), ("WWWW", 6, False), ("WWWWW", 1, False),
                                              ("W", 7, False)])
def test_every_schedule_is_ordered(units, slices, tma, overlap):
    for seed in range(25):
        run(units, slices, tma, overlap, seed)
        run(units, slices, tma, overlap, seed, slow=(4, 5, 6, 7) if not tma else (1,))


def _caught(drop, tma, slow=(), units="WWWH", slices=6, seeds=40):
    n = 0
    for seed in range(seeds):
        try:
            run(units if tma else units.replace("H", "W"), slices, tma, 96, seed, drop, slow)
        except AssertionError:
            n += 1
    return n


@pytest.mark.parametrize("tma", [True, False])
@pytest.mark.parametrize("drop", ["empty", "full", "scales", "shared", "tfull"])
def test_a_missing_wait_is_caught(drop, tma):
    assert _caught(drop, tma) >= 10


def test_the_accumulators_wait():
    """Needed without TMA stores, where only four warps say that the shared columns are free
    (slow others show it); implied with them."""
    assert _caught("drained", False, slow=(4, 5, 6, 7, 12, 13, 14, 15), units="WWWWW", slices=1) >= 10
    assert _caught("drained", True, slow=(1, 6), units="WWWWH", slices=1) == 0
    assert _caught("drained", True, units="WWWWW", slices=2) == 0
