"""A randomised model of the barrier protocol of the 8-bit cache's attention for many rows
(`prompt_kernel` in the attention kernels).

Roles of a CTA: one producer (K and V stages and the tiles' scale slots), one V converter,
two softmax groups and two MMA issuers (one a 128-row Q tile each).  A share is a list of
units, each with one or two Q tiles that hold rows and some K, V tiles; every role walks the
same list.  The model replays the waits and arrivals with the hardware's parity semantics
(`Bar.try_wait` also checks the true phase) under random interleavings and latencies of
copies and matrix products, and tracks what each buffer holds.  It fails on a wait that a
wrong phase satisfies, on a product that reads another tile's operands, on scores or weights
that overwrite ones still to be read, on a scale slot refilled too early, and on a deadlock.

The variant in which an issuer whose Q tile holds no rows lets the stages of that unit pass
without observing them fails: it comes back more than one phase ahead of a stage's barrier
and takes an older phase for its own."""
import random

import pytest

from test_pipeline_protocol import Bar

KST, VST, CST, SLOTS = 4, 3, 3, 8


def simulate(seed, units, observe=True, slots=SLOTS):
    rnd = random.Random(seed)
    kfull, kempty = [Bar(1) for _ in range(KST)], [Bar(2) for _ in range(KST)]
    vfull, vempty = [Bar(1) for _ in range(VST)], [Bar(1) for _ in range(VST)]
    cfull, cempty = [Bar(1) for _ in range(CST)], [Bar(2) for _ in range(CST)]
    qfull, sfull, sread, pread, ofull = ([Bar(1) for _ in range(2)] for _ in range(5))
    pfull = [[Bar(1), Bar(1)] for _ in range(2)]
    k_held, v_held, c_held, slot_held = [None] * KST, [None] * VST, [None] * CST, [None] * slots
    s_held, p_held = [None, None], [[None, None], [None, None]]   # the tiles in S_t's columns and in P_t's two parts
    clock, events = [0], []
    queue = [[], []]                 # each issuer's products and commits, executed in order

    def later(fn):
        events.append((clock[0] + rnd.randint(1, 30), fn))

    def producer():
        n = 0
        for act, tiles in units:
            for _ in range(tiles):
                ks, vs = n % KST, n % VST
                while not kempty[ks].try_wait(n // KST - 1) if n >= KST else False:
                    yield
                slot_held[n % slots] = n
                kfull[ks].arrive(tx=1)

                def land_k(ks=ks, n=n):
                    k_held[ks] = n
                    kfull[ks].complete_tx(1)
                later(land_k)
                yield
                while not vempty[vs].try_wait(n // VST - 1) if n >= VST else False:
                    yield
                vfull[vs].arrive(tx=1)

                def land_v(vs=vs, n=n):
                    v_held[vs] = n
                    vfull[vs].complete_tx(1)
                later(land_v)
                n += 1
                yield

    def converter():
        n = 0
        for act, tiles in units:
            for _ in range(tiles):
                vs, vb = n % VST, n % CST
                while not vfull[vs].try_wait(n // VST):
                    yield
                assert v_held[vs] == n and slot_held[n % slots] == n
                yield
                assert v_held[vs] == n
                vempty[vs].arrive()
                while not cempty[vb].try_wait(n // CST - 1) if n >= CST else False:
                    yield
                assert slot_held[n % slots] == n, "the tile's scales were overwritten"
                c_held[vb] = n
                yield
                cfull[vb].arrive()
                n += 1

    def softmax(t):
        n = ns = 0
        for act, tiles in units:
            if t >= act:
                n += tiles
                continue
            yield
            qfull[t].arrive()
            for j in range(tiles):
                while not sfull[t].try_wait(ns):
                    yield
                assert s_held[t] == n, (s_held[t], n)
                assert slot_held[n % slots] == n, "the tile's scales were overwritten"
                yield
                assert s_held[t] == n
                s_held[t] = None                     # read
                sread[t].arrive()
                yield
                correct = j and rnd.random() < 0.3
                for half in range(2):
                    for _ in range(rnd.randint(1, 3)):
                        yield
                    if j:                            # the accumulator is corrected, or this part's place is free
                        while not (ofull if half or correct else pread)[t].try_wait(ns - 1):
                            yield
                    assert p_held[t][half] is None, "weights still being read"
                    assert not correct or half or p_held[t][1] is None
                    p_held[t][half] = n
                    pfull[t][half].arrive()
                n, ns = n + 1, ns + 1
            while not ofull[t].try_wait(ns - 1):
                yield

    def issuer(t):
        n = nq = np = 0

        def scores(n):
            def run():
                assert k_held[n % KST] == n, "scores of another tile's keys"
                assert s_held[t] is None, "scores over scores that were not read"
                s_held[t] = n
            queue[t].append(run)
            queue[t].append(sfull[t].arrive)
            queue[t].append(kempty[n % KST].arrive)

        def values(n, half):
            def run():
                assert c_held[n % CST] == n, "weights times another tile's values"
                assert p_held[t][half] == n, (p_held[t], n, half)
                p_held[t][half] = None
            queue[t].append(run)
            if not half:
                queue[t].append(pread[t].arrive)
            else:
                queue[t].append(ofull[t].arrive)
                queue[t].append(cempty[n % CST].arrive)
        for act, tiles in units:
            if t >= act:
                for _ in range(tiles):
                    if observe:
                        while not kfull[n % KST].try_wait(n // KST):
                            yield
                        kempty[n % KST].arrive()
                        while not cfull[n % CST].try_wait(n // CST):
                            yield
                        cempty[n % CST].arrive()
                    else:                            # the other issuer arrives twice instead
                        queue[t].append(kempty[n % KST].arrive)
                        queue[t].append(cempty[n % CST].arrive)
                    n += 1
                continue
            while not qfull[t].try_wait(nq):
                yield
            nq += 1
            while not kfull[n % KST].try_wait(n // KST):
                yield
            scores(n)
            for j in range(tiles):
                while not sread[t].try_wait(np):
                    yield
                if j + 1 < tiles:
                    while not kfull[(n + 1) % KST].try_wait((n + 1) // KST):
                        yield
                    scores(n + 1)
                for half in range(2):
                    while not pfull[t][half].try_wait(np):
                        yield
                    if half == 0:
                        while not cfull[n % CST].try_wait(n // CST):
                            yield
                    values(n, half)
                n, np = n + 1, np + 1
                yield

    live = [producer(), converter(), softmax(0), softmax(1), issuer(0), issuer(1)]
    total, steps = sum(x for _, x in units), 0
    while live or queue[0] or queue[1]:
        steps += 1
        if steps > 20_000 + 4_000 * total:
            raise AssertionError("deadlock")
        events.sort(key=lambda e: e[0])
        if events and rnd.random() < 0.3:
            at, fn = events.pop(0)
            clock[0] = max(clock[0], at)
            fn()
            continue
        t = rnd.randint(0, 1)
        if queue[t] and rnd.random() < 0.4:
            queue[t].pop(0)()
            continue
        if not live:
            continue
        r = rnd.choice(live)
        clock[0] += 1
        try:
            next(r)
        except StopIteration:
            live.remove(r)


def some_units(rnd):
    return [(rnd.randint(1, 2), rnd.randint(1, 9)) for _ in range(rnd.randint(1, 6))]


def test_random_shares():
    for seed in range(120):
        simulate(seed, some_units(random.Random(seed)))


@pytest.mark.parametrize("units", [[(1, 1)], [(2, 1)], [(1, 20), (2, 5)], [(2, 3), (1, 14), (2, 2), (1, 1), (2, 9)]])
def test_units_with_and_without_a_second_tile(units):
    for seed in range(30):
        simulate(seed, units)


def _failures(**kw):
    bad = 0
    for seed in range(40):
        try:
            simulate(seed, [(2, 3), (1, 14), (2, 6), (1, 9), (2, 5)], **kw)
        except AssertionError:
            bad += 1
    return bad


def test_model_catches_an_issuer_that_does_not_observe_a_unit():
    assert _failures(observe=False) > 10


def test_model_catches_too_few_scale_slots():
    assert _failures(slots=3) > 10
