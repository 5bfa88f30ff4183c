"""A randomised model of one Q tile's softmax group and MMA issuer in the 8-bit cache's attention
for many rows, with the loop that a unit's part goes on in from a tile whose value scales lie apart.

The ordinary loop releases the scores as soon as they are read, then waits for the places of the
weights; the other waits for the accumulator first, hands over a tile's weights at once and
releases its scores with them.  A share is a list of units (tiles, the tile from which the second
loop takes over).  Keys and values are always there: their stages are modelled elsewhere.  The model
fails on a wait that a wrong phase satisfies (`Bar.try_wait` checks the true phase), on scores or
weights that are overwritten before they are read, on an accumulator that is read or corrected while a
product runs, and on a deadlock."""
import random

import pytest

from test_pipeline_protocol import Bar


def simulate(seed, units, early=False):
    rnd = random.Random(seed)
    qfull, sfull, sread, pread, ofull = (Bar(1) for _ in range(5))
    pfull = [Bar(1), Bar(1)]
    scores, weights = [None], [None, None]   # the tiles in the score columns and in the weights' two parts
    queue = []                               # products and commits, executed in order
    touching = [False]                       # the softmax group is at the accumulator

    def softmax():
        ns = 0
        for tiles, apart in units:
            yield
            qfull.arrive()
            for j in range(tiles):
                while not sfull.try_wait(ns):
                    yield
                assert scores[0] == ns
                yield
                if j < apart:                # the ordinary loop
                    scores[0] = None
                    sread.arrive()
                    yield
                    correct = j and rnd.random() < 0.3
                    for half in range(2):
                        if j:
                            while not (ofull if half or correct else pread).try_wait(ns - 1):
                                yield
                        if correct and not half:
                            touching[0] = True
                            yield
                            touching[0] = False
                        assert weights[half] is None
                        weights[half] = ns
                        pfull[half].arrive()
                        yield
                else:
                    if j and not early:
                        while not ofull.try_wait(ns - 1):
                            yield
                    if j and rnd.random() < 0.5:
                        touching[0] = True
                        yield
                        touching[0] = False
                    assert scores[0] == ns, "scores overwritten before the weights were formed"
                    for half in range(2):
                        assert weights[half] is None, "weights still being read"
                        weights[half] = ns
                        yield
                    assert scores[0] == ns
                    scores[0] = None
                    for bar in (sread, pfull[0], pfull[1]):
                        bar.arrive()
                        if rnd.random() < 0.5:
                            yield
                ns += 1
            while not ofull.try_wait(ns - 1):
                yield
            touching[0] = True               # the results are read
            yield
            touching[0] = False

    def issuer():
        n = nq = 0

        def first(n):
            def run():
                assert scores[0] is None, "scores over scores that were not read"
                scores[0] = n
            queue.extend([run, sfull.arrive])

        def second(n, half):
            def run():
                assert weights[half] == n and not touching[0]
                weights[half] = None
            queue.extend([run, (ofull if half else pread).arrive])
        for tiles, _ in units:
            while not qfull.try_wait(nq):
                yield
            nq += 1
            first(n)
            for j in range(tiles):
                while not sread.try_wait(n):
                    yield
                if j + 1 < tiles:
                    first(n + 1)
                for half in range(2):
                    while not pfull[half].try_wait(n):
                        yield
                    second(n, half)
                n += 1
                yield

    live, steps, total = [softmax(), issuer()], 0, sum(t for t, _ in units)
    while live or queue:
        steps += 1
        assert steps < 5_000 + 2_000 * total, "deadlock"
        if queue and rnd.random() < 0.4:
            queue.pop(0)()
            continue
        if not live:
            continue
        r = rnd.choice(live)
        try:
            next(r)
        except StopIteration:
            live.remove(r)


@pytest.mark.parametrize("units", [[(1, 0)], [(5, 0)], [(5, 2)], [(5, 5), (4, 0), (1, 1), (3, 1)], [(1, 0), (6, 3), (7, 7), (2, 1)]])
def test_parts_that_change_over(units):
    for seed in range(60):
        simulate(seed, units)


def test_random_parts():
    for seed in range(150):
        rnd = random.Random(seed)
        units = [(t, rnd.randint(0, t)) for t in (rnd.randint(1, 9) for _ in range(rnd.randint(1, 6)))]
        simulate(seed, units)


def test_model_catches_weights_written_before_the_accumulator_is_at_rest():
    bad = 0
    for seed in range(40):
        try:
            simulate(seed, [(6, 0), (5, 2)], early=True)
        except AssertionError:
            bad += 1
    assert bad > 10
