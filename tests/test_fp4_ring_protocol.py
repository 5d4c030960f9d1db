"""A randomized CPU model of the rings that the 4-bit quantizer and the block norm stream their
rows through: W warps of a CTA take every row together, one thread copies the next rows into S
slots, and a row has one or two block barriers.  A slot's `full` mbarrier takes one arrival and
the copy's bytes a phase.

Some copies land late, and a warp's wait may give up before they do.  Then no slot may be
filled again while a copy into it is in flight, no barrier may get an arrival that its phase has
no place for, every warp has to reach every block barrier (one left alone would wait for good),
and the CTA must not end with a copy in flight, for its shared memory may be the next CTA's by
then.

The rule: a wait that gives up raises a flag in front of a block barrier; behind it the copying
thread fills no slot while the flag is up, all warps go on with the rows as they are, and the
copying thread stays at the end until the copies in flight have landed."""
import random

import pytest


class Broken(AssertionError):
    pass


class MBarrier:
    def __init__(self):
        self.pending, self.tx, self.phases = 1, 0, 0

    def _check(self):
        if self.pending == 0 and self.tx == 0:
            self.phases += 1
            self.pending = 1

    def arrive_expect(self, tx):
        self.tx += tx
        self.pending -= 1
        if self.pending < 0:
            raise Broken("arrival beyond the barrier's count")
        self._check()

    def complete(self, tx):
        self.tx -= tx
        self._check()

    def passed(self, parity):
        return (self.phases & 1) != parity


def run(warps, slots, rows, barriers, seed, late=0.0, form="mended"):
    """One schedule; True if a wait gave up.  late: share of the copies that outlast a wait.
    Forms: "mended"; "refilling": slots are filled again whatever the waits gave; "no hold": the
    CTA leaves at once."""
    rng = random.Random(seed)
    full = [MBarrier() for _ in range(slots)]
    holds = [None] * slots
    landing = []                       # [slot, row, steps to go]
    raised = [False]
    count, generation = [0], [0]       # the block barrier

    def fetch(row, s):
        if any(c[0] == s for c in landing):
            raise Broken("a copy into a slot that one is still in flight to")
        full[s].arrive_expect(1)
        holds[s] = None
        landing.append([s, row, rng.randrange(200, 900) if rng.random() < late else rng.randrange(1, 30)])

    def wait(s, phase):
        """False after a limited time, or soon after another wait has given up."""
        polls = 0
        while not full[s].passed(phase):
            polls += 1
            if polls > (2 if raised[0] else 60):
                raised[0] = True
                return False
            yield
        return True

    def barrier():
        mine = generation[0]
        count[0] += 1
        if count[0] == warps:
            count[0] = 0
            generation[0] += 1
        while generation[0] == mine:
            yield

    def warp(w):
        if w == 0:
            for row in range(min(slots, rows)):
                fetch(row, row)
        yield from barrier()
        s = phase = 0
        for row in range(rows):
            ok = yield from wait(s, phase)
            if ok and not raised[0] and holds[s] != row:
                raise Broken("a row read from a slot that does not hold it")
            yield
            for _ in range(barriers):
                yield from barrier()
                yield
            if w == 0 and row + slots < rows and (form == "refilling" or not raised[0]):
                fetch(row + slots, s)
            s, phase = (0, phase ^ 1) if s + 1 == slots else (s + 1, phase)
            yield
        if w == 0 and raised[0] and form != "no hold":
            for _ in range(1000):
                yield

    agents = {w: warp(w) for w in range(warps)}
    weight = [rng.choice((1, 1, 4, 40)) for _ in range(warps)]
    for _ in range(60000):
        if not agents:
            if landing:
                raise Broken("the CTA ends with a copy in flight")
            return raised[0]
        for c in landing:
            c[2] -= 1
        for c in [c for c in landing if c[2] <= 0]:
            landing.remove(c)
            holds[c[0]] = c[1]
            full[c[0]].complete(1)
        live = list(agents)
        w = rng.choices(live, [weight[k] for k in live])[0]
        try:
            next(agents[w])
        except StopIteration:
            del agents[w]
    raise Broken("a warp waits for good")


SHAPES = [(1, 2, 9, 1), (4, 2, 9, 1), (4, 3, 11, 2), (8, 2, 7, 2), (2, 6, 15, 2)]


@pytest.mark.parametrize("warps,slots,rows,barriers", SHAPES)
def test_every_schedule_ends(warps, slots, rows, barriers):
    stops = 0
    for seed in range(80):
        run(warps, slots, rows, barriers, seed)
        stops += run(warps, slots, rows, barriers, seed, late=0.15)
    assert stops > 10, "the schedules reach the case"


@pytest.mark.parametrize("form", ["refilling", "no hold"])
def test_leaving_a_part_out_is_caught(form):
    caught = 0
    for seed in range(200):
        try:
            run(4, 2, 9, 1, seed, late=0.15, form=form)
        except Broken:
            caught += 1
    assert caught > 3, f"{form}: {caught}"
