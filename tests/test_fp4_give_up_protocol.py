"""A randomized CPU model of how the 4-bit GEMM kernels end when a wait gives up: a CTA's producer
with its ring of stages, the issuing thread and the epilogue, and loads that may land long after
a wait for them has run out.  The CTA must not end with a load in flight: its shared memory may
be another CTA's by then.

The producer may have issued its last loads, and be done, when the issuing thread gives up on
one of them.  So not the producer's own waits say whether the CTA has to stay: at the block
barrier that everybody reaches the flag of any wait that gave up is final, and behind it one
thread, finding it up, stays until the loads in flight have landed.

Nor may tensor memory be released, behind that barrier, with products in flight, as they may be
when the issuing thread or the epilogue gives up, on a load or because another warp has: the
issuing thread waits for its own in any case."""
import random

import pytest


class Broken(AssertionError):
    pass


def run(slices, stages, seed, late=0.0, form="mended"):
    """One schedule; True if a wait gave up.  Forms: "mended"; "producer": the producer stays if a
    wait of its own gave up, and nobody else; "early": the flag is read before the barrier;
    "issuer": the issuing thread does not wait for its products."""
    rng = random.Random(seed)
    full, empty = [0] * stages, [0] * stages           # completed phases
    tfull = [0]
    landing, queue = [], []
    raised, here = [False], [0]

    def wait(done):
        polls = 0
        while not done():
            polls += 1
            if polls > (2 if raised[0] else 150):
                raised[0] = True
                return False
            yield
        return True

    def hold():
        for _ in range(3000):
            yield

    def barrier(who):
        if form == "early" and who == "producer" and raised[0]:
            yield from hold()
        here[0] += 1
        while here[0] < 3:
            yield
        if form in ("mended", "issuer") and who == "producer" and raised[0]:
            yield from hold()

    def other():
        """Another warp's wait gives up, at any time."""
        for _ in range(rng.randrange(10, 400)):
            yield
        raised[0] = True

    def producer():
        ok = True
        for it in range(slices):
            s, n = it % stages, it // stages
            ok = yield from wait(lambda: empty[s] >= n)
            if not ok:
                break
            landing.append([s, rng.randrange(800, 2500) if rng.random() < late else rng.randrange(1, 40)])
            yield
        if not ok and form == "producer":
            yield from hold()
        yield from barrier("producer")

    def issuer():
        for it in range(slices):
            s, n = it % stages, it // stages
            if not (yield from wait(lambda: full[s] > n)):
                break
            queue.append(("empty", s))
            if it == slices - 1:
                queue.append(("tfull", 0))
            yield
        while queue and form != "issuer":
            yield
        yield from barrier("issuer")
        if queue:
            raise Broken("tensor memory released with products in flight")

    def epilogue():
        yield from wait(lambda: tfull[0] > 0)
        yield from barrier("epilogue")

    agents = [producer(), issuer(), epilogue()] + ([other()] if late and rng.random() < 0.5 else [])
    weights = [rng.choice((1, 1, 4)) for _ in agents]
    pipe = rng.choice((0.3, 0.3, 0.01))
    for _ in range(60000):
        if not agents:
            if landing:
                raise Broken("the CTA ends with a load in flight")
            return raised[0]
        for c in landing:
            c[1] -= 1
        for c in [c for c in landing if c[1] <= 0]:
            landing.remove(c)
            full[c[0]] += 1
        if queue and rng.random() < pipe:
            kind, s = queue.pop(0)
            if kind == "empty":
                empty[s] += 1
            else:
                tfull[0] += 1
        k = rng.choices(range(len(agents)), weights)[0]
        try:
            next(agents[k])
        except StopIteration:
            del agents[k], weights[k]
    raise Broken("a warp waits for good")


@pytest.mark.parametrize("slices,stages", [(1, 5), (4, 5), (5, 5), (12, 5), (9, 3)])
def test_every_schedule_ends(slices, stages):
    stops = 0
    for seed in range(60):
        run(slices, stages, seed)
        stops += run(slices, stages, seed, late=0.2)
    assert stops > 5, "the schedules reach the case"


@pytest.mark.parametrize("form", ["producer", "early", "issuer"])
def test_another_form_is_caught(form):
    caught = 0
    for seed in range(100):
        try:
            run(4, 5, seed, late=0.2, form=form)
        except Broken:
            caught += 1
    assert caught > 5, f"{form}: {caught}"
