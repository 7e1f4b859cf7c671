"""The barriers of the quantised-cache decode kernel, as a model run under random schedules.

The kernel's producers (K, V) fill a ring of stages by asynchronous copies that land in
any order; its consumer warps take units of the stages in turn, so a warp meets a slot only
in some of its turns.  Barriers are waited for by the parity of a phase, as on the device: a
phase two behind passes for one that is done.  The model checks that no slot is read before
its data or written while it is read, that no barrier gets too many arrivals, and that
every warp ends.
"""
import random

import pytest

WARPS = 8


class Barrier:
    def __init__(self, count):
        self.count, self.pending, self.phase, self.bytes = count, count, 0, 0

    def arrive(self, n_bytes=0):
        self.bytes += n_bytes
        self.pending -= 1
        assert self.pending >= 0, "more arrivals than a phase has"
        self.settle()

    def landed(self):
        self.bytes -= 1
        self.settle()

    def settle(self):
        if self.pending == 0 and self.bytes == 0:
            self.pending, self.phase = self.count, self.phase + 1

    def done(self, parity):
        return (self.phase & 1) != parity


def run(segments, stages, units_per_stage, rng, look_at_empty=True):
    """One CTA; segments: its blocks of each (sequence, KV head)."""
    full = [Barrier(2) for _ in range(stages)]
    empty = [Barrier(units_per_stage) for _ in range(stages)]
    copies, reading, joins = [], [0] * stages, {}

    def producer():
        issued, free = 0, True
        for _ in range(sum(segments)):
            slot, turn = issued % stages, issued // stages
            while not free:
                yield
                free = empty[slot].done((turn - 1) & 1)
            assert reading[slot] == 0, "written while it is read"
            full[slot].arrive(2)
            copies.extend([slot, slot])
            issued += 1
            yield
            free = issued < stages or empty[issued % stages].done((issued // stages - 1) & 1)
        for i in range(max(issued - stages, 0), issued):
            while not full[i % stages].done((i // stages) & 1):
                yield

    def join(key, active):
        joins[key] = joins.get(key, 0) + 1
        assert joins[key] <= active
        while joins[key] < active:
            yield

    def consumer(warp):
        unit = stage0 = 0
        for k, n in enumerate(segments):
            units = n * units_per_stage
            first, active = (warp - unit) % WARPS, min(units, WARPS)
            last = 0
            for u in range(first, units, WARPS):
                last = (stage0 + u // units_per_stage) % stages
                slot, turn = last, (stage0 + u // units_per_stage) // stages
                while look_at_empty and turn > 0 and not empty[slot].done((turn - 1) & 1):
                    yield
                while not full[slot].done(turn & 1):
                    yield
                assert full[slot].phase == turn + 1, "read before its data"
                reading[slot] += 1
                yield
                reading[slot] -= 1
                if u + WARPS < units:
                    empty[slot].arrive()
                yield
            if first < units:
                yield from join((k, 0), active)
                yield from join((k, 1), active)
                empty[last].arrive()   # the last stage only after the join
            unit += units
            stage0 += n
            yield

    warps = [producer(), producer()] + [consumer(w) for w in range(WARPS)]
    live, steps = list(range(len(warps))), 0
    speed, landing = [], rng.choice([0.01, 0.05, 0.3, 1.0])
    while live:
        if steps % 2000 == 0:
            speed = [rng.random() ** 3 + 0.001 for _ in warps]
        steps += 1
        assert steps < 400000, "warps that never end"
        if copies and rng.random() < landing:
            full[copies.pop(rng.randrange(len(copies)))].landed()
        w = rng.choices(live, [speed[i] for i in live])[0]
        try:
            next(warps[w])
        except StopIteration:
            live.remove(w)
    assert not copies


# (stages, units of a stage) of the supported head sizes, block sizes and bits
RINGS = [(14, 1), (14, 2), (14, 4), (12, 4), (11, 2), (10, 4), (8, 4), (5, 4), (4, 4), (9, 2), (4, 8), (2, 8)]
SHAPES = [[30], [1] * 40, [13, 14], [2, 7, 1, 1, 20, 3]]


@pytest.mark.parametrize("stages,units", RINGS)
def test_ring_of_the_decode_kernel(stages, units):
    rng = random.Random(stages * 100 + units)
    for segments in SHAPES:
        for _ in range(3):
            run(segments, stages, units, rng)


def test_the_model_finds_a_parity_that_passes_for_another():
    # without a look at the slot's last turn, a phase still open can pass for the next one
    rng = random.Random(1)
    with pytest.raises(AssertionError, match="read before its data"):
        for _ in range(200):
            run([14], 5, 4, rng, look_at_empty=False)
