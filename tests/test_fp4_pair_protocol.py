"""A randomized CPU model of the synchronisation of the 4-bit GEMM's pair kernel: two CTAs'
producers, the even CTA's issuing thread, the tensor pipe, and both CTAs' epilogue warps,
with the kernel's barriers, ring of slots, two sets of scale columns and two accumulators that
share columns.

What the hardware orders is all that the model orders: products run in issue order; a scale
copy runs before the products issued after it, at any time, even ahead of products issued
before it; a commit arrives when everything issued before it is done; a load lands at any
time.  Under random schedules a product must find its own slice in both CTAs' slots and in
the scale columns, must not write columns that an epilogue warp still has to read, and an
epilogue warp must find its own tile.  Leaving out any one of the waits must be caught."""
import random

import pytest

STAGES = 5


class MBarrier:
    def __init__(self, count):
        self.count = self.pending = count
        self.tx = 0
        self.phases = 0

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.phases += 1
            self.pending = self.count

    def arrive(self, tx=0):
        self.tx += tx
        self.pending -= 1
        assert self.pending >= 0, "arrival beyond the barrier's count"
        self._check()

    def complete(self, tx):
        self.tx -= tx
        self._check()

    def passed(self, parity):
        return (self.phases & 1) != parity


def run(tiles, slices, parts, seed, drop=()):
    rng = random.Random(seed)
    warps = 4 * parts
    full = [MBarrier(1) for _ in range(STAGES)]
    empty = [[MBarrier(1) for _ in range(STAGES)] for _ in range(2)]
    tfull = [[MBarrier(1), MBarrier(1)] for _ in range(2)]
    tshared = MBarrier(8)
    tdrained = [MBarrier(2 * warps), MBarrier(2 * warps)]
    slots = [[None] * STAGES for _ in range(2)]
    scales = [None, None]                    # slice whose scales a set of columns holds
    # columns: low accumulator only, shared, high accumulator only
    owner = {"low": None, "shared": None, "high": None}
    unread = {r: set() for r in owner}       # (cta, warp) that still have to read a region
    of_tile = lambda i: ("low", "shared") if i % 2 == 0 else ("shared", "high")  # noqa: E731

    def readers(i, region):
        """Warps of a CTA that read a region of tile i's accumulator."""
        if parts == 1:
            return range(4)
        if region == "shared":               # the last columns of the lower, the first of the upper one
            return range(4, 8) if i % 2 == 0 else range(4)
        return range(8)                      # both halves of the columns reach into the rest

    landing, queue, cps = [], [], []         # loads in flight; issued products and commits; copies
    done = {"mma": -1}

    def producer(cta):
        it = 0
        for _ in range(tiles):
            for _ in range(slices):
                s, ph = it % STAGES, (it // STAGES) & 1
                while not empty[cta][s].passed(ph ^ 1):
                    yield
                if cta == 0:
                    full[s].arrive(tx=2)
                landing.append((cta, s, it))
                it += 1
                yield

    def issuer():
        it = 0
        for i in range(tiles):
            if i > 1 and "drained" not in drop:
                while not tdrained[i & 1].passed(((i >> 1) - 1) & 1):
                    yield
            if i > 0 and "shared" not in drop:
                while not tshared.passed((i - 1) & 1):
                    yield
            for ks in range(slices):
                s, ph = it % STAGES, (it // STAGES) & 1
                if it >= 2 and "scales" not in drop:
                    while not empty[0][(it - 2) % STAGES].passed(((it - 2) // STAGES) & 1):
                        yield
                if "full" not in drop:
                    while not full[s].passed(ph):
                        yield
                cps.append(it)
                queue.append(("mma", it, i, ks))
                queue.append(("commit", [empty[0][s], empty[1][s]]))
                if ks == slices - 1:
                    queue.append(("commit", [tfull[0][i & 1], tfull[1][i & 1]]))
                it += 1
                yield

    def copy_scales():
        it = cps.pop(0)
        assert done["mma"] >= it - 2, "scales replaced before the products that use them"
        for cta in range(2):
            assert slots[cta][it % STAGES] == it, "scales of another slice copied"
        scales[it & 1] = it

    def tensor():
        while True:
            if queue:
                op = queue[0]
                if op[0] == "commit":
                    for bar in op[1]:
                        bar.arrive()
                else:
                    _, it, i, ks = op
                    while cps and cps[0] <= it:
                        copy_scales()
                    if ks == 0:
                        for region in of_tile(i):
                            assert not unread[region], "columns written before they were read"
                            owner[region] = i
                    for k in range(4):                       # a product of several steps
                        for cta in range(2):
                            assert slots[cta][it % STAGES] == it, "product of another slice"
                        assert scales[it & 1] == it, "product with another slice's scales"
                        if k < 3:
                            yield
                    if ks == slices - 1:
                        for region in of_tile(i):
                            assert owner[region] == i
                            unread[region] = {(c, w) for c in range(2) for w in readers(i, region)}
                    done["mma"] = it
                queue.pop(0)
            yield

    def epilogue(cta, w):
        for i in range(tiles):
            buf = i & 1
            while not tfull[cta][buf].passed((i >> 1) & 1):
                yield
            mine = [r for r in of_tile(i) if w in readers(i, r)]
            for region in sorted(mine, key=lambda r: r != "shared"):
                assert owner[region] == i, "accumulator of another tile"
                unread[region].discard((cta, w))
                if region == "shared":
                    yield
                    tshared.arrive()
                yield
            tdrained[buf].arrive()
            yield

    actors = [producer(0), producer(1), issuer()] + [epilogue(c, w) for c in range(2) for w in range(warps)]
    weights = [rng.choice((1, 1, 3, 10)) for _ in actors]
    pipe = tensor()
    speed = rng.choice((0.02, 0.08, 0.25))                   # of the tensor pipe
    alive = list(range(len(actors)))
    for _ in range(400000):
        if not alive:
            return
        x = rng.random()
        if x < speed:
            next(pipe)
        elif x < 0.4 and landing:
            cta, s, it = landing.pop(rng.randrange(len(landing)))
            slots[cta][s] = it
            full[s].complete(1)
        elif x < 0.45 and cps:
            copy_scales()                                    # ahead of earlier products
        else:
            a = rng.choices(alive, [weights[k] for k in alive])[0]
            try:
                next(actors[a])
            except StopIteration:
                alive.remove(a)
    raise RuntimeError("no progress")


@pytest.mark.parametrize("parts", [1, 2])
@pytest.mark.parametrize("tiles,slices", [(1, 1), (2, 1), (5, 1), (3, 2), (6, 3), (4, 7), (3, 12)])
def test_every_schedule_is_ordered(parts, tiles, slices):
    for seed in range(40):
        run(tiles, slices, parts, seed)


@pytest.mark.parametrize("drop,parts", [("shared", 1), ("shared", 2), ("scales", 1), ("full", 1), ("drained", 2)])
def test_a_missing_wait_is_caught(drop, parts):
    caught = 0
    for seed in range(60):
        try:
            run(4, 6, parts, seed, drop=(drop,))
        except AssertionError:
            caught += 1
    assert caught, drop
