"""How the shared tokens' pass divides its units (EvenUnits in the attention kernels), modelled on
the host.

A CTA walks the units that its share of the costs touches, as prompt_kernel does, or takes one part
of one unit; the join finds a unit's parts by arithmetic.  Every token tile of every unit is taken
once, parts of a unit lie in consecutive CTAs with tiles in each, a CTA holds at most one part begun
before its share and one that goes on after it, and the join finds the CTAs that hold tiles."""
import random

import pytest

UNIT_TILES, ROWS = 6, 256


class Even:
    def __init__(self, pairs, heads, tokens, d, most):
        n = 80 if d == 128 else 128
        self.n_kv = -(-tokens // n)
        self.units = -(-pairs // ROWS) * heads if self.n_kv else 0
        self.cost, self.parts, self.n_cta = self.n_kv + UNIT_TILES, 0, 0
        self.total = self.units * self.cost
        if not self.units:
            return
        self.n_cta = min(most, (self.total + UNIT_TILES + 1) // (UNIT_TILES + 2))
        if self.units <= most and self.total <= 12 * self.n_cta:
            k = min(most * 2 // 3 // self.units, (self.n_kv + 2) // 3)
            if k > 0 and 3 * -(-self.n_kv // k) <= 2 * -(-self.total // self.n_cta):
                self.parts, self.n_cta = k, self.units * k

    def find(self, unit):
        if self.parts:
            return unit * self.parts, self.parts
        first = ((unit * self.cost + UNIT_TILES + 1) * self.n_cta - 1) // self.total
        return first, ((unit + 1) * self.cost * self.n_cta - 1) // self.total - first + 1


def walk(e, cta):
    """(unit, j0, j1) of a CTA's parts."""
    if e.parts:
        unit, i = divmod(cta, e.parts)
        return [(unit, e.n_kv * i // e.parts, e.n_kv * (i + 1) // e.parts)]
    a, b = e.total * cta // e.n_cta, e.total * (cta + 1) // e.n_cta
    unit, at = divmod(a, e.cost)
    left, parts = b - a, []
    while left > 0:
        to = min(e.cost, at + left)
        j0, j1 = max(0, at - UNIT_TILES), max(0, to - UNIT_TILES)
        if j1 <= j0:
            assert not parts or j1 == 0
            break
        parts.append((unit, j0, j1))
        left -= to - at
        at, unit = 0, unit + 1
    return parts


@pytest.mark.parametrize("seed", range(12))
def test_every_tile_once_and_found_again(seed):
    rnd = random.Random(seed)
    kinds = set()
    for _ in range(80):
        log = lambda hi: int(round(hi ** rnd.random()))  # noqa: E731
        e = Even(log(5000), rnd.choice([1, 2, 3, 4, 8, 32]), log(30000), rnd.choice([64, 128]), rnd.choice([1, 7, 152]))
        kinds.add(e.parts > 0)
        taken = {}
        for cta in range(e.n_cta):
            parts = walk(e, cta)
            for i, (unit, j0, j1) in enumerate(parts):
                assert j1 > j0 and (i == 0 or j0 == 0) and (i == len(parts) - 1 or j1 == e.n_kv)
                for j in range(j0, j1):
                    assert (unit, j) not in taken
                    taken[unit, j] = cta
        assert len(taken) == e.units * e.n_kv
        for unit in range(e.units):
            first, n = e.find(unit)
            assert [first + i for i in range(n)] == sorted({taken[unit, j] for j in range(e.n_kv)})
    assert kinds == {False, True}
