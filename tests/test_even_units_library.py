"""The division of the shared tokens' pass as the library computes it (EvenUnits, through a testing
hook) against the model of test_even_units.py, whose numbers have no width."""
import random

import pytest

from test_even_units import Even, walk
from test_serve_abi import kvrp  # noqa: F401

MOST_TOKENS = 0x7fffff00


def _compare(kvrp, pairs, heads, tokens, d, most, rnd):  # noqa: F811
    e = Even(pairs, heads, tokens, d, most)
    units = sorted({0, e.units - 1, *(rnd.randrange(e.units) for _ in range(40))}) if e.units else []
    blocks = sorted({0, e.n_cta - 1, *(rnd.randrange(e.n_cta) for _ in range(40))}) if e.n_cta else []
    shape, found, ends = kvrp.kvrp_test_even_units(pairs, heads, tokens, head_dim=d, most_cta=most, units=units, blocks=blocks)
    assert shape == (e.n_kv, e.parts, e.units, e.cost, e.n_cta)
    assert found == [e.find(u) for u in units]
    for b, (begin, end) in zip(blocks, ends):
        if e.parts:
            assert walk(e, b) == [(b // e.parts, begin, end)]
        else:
            assert (begin, end) == (e.total * b // e.n_cta, e.total * (b + 1) // e.n_cta)
    return e


@pytest.mark.parametrize("seed", range(8))
def test_like_the_model(kvrp, seed):  # noqa: F811
    rnd = random.Random(seed)
    log = lambda hi: int(round(hi ** rnd.random()))  # noqa: E731
    kinds = set()
    for _ in range(150):
        e = _compare(kvrp, log(5000), rnd.choice([1, 2, 3, 4, 8, 32]), log(200000), rnd.choice([64, 128]), rnd.choice([1, 7, 152]), rnd)
        kinds.add(e.parts > 0)
    assert kinds == {False, True}


@pytest.mark.parametrize("heads", [1, 3, 16, 17, 255, 4096])
@pytest.mark.parametrize("d", [64, 128])
def test_at_the_limits(kvrp, heads, d):  # noqa: F811
    """As many (row, query head) pairs as the call takes (rows x group below 2^28, rows x query heads below 2^32), and as
    many tokens."""
    rnd = random.Random(heads)
    most = min((1 << 28) - 257, ((1 << 32) - 1) // heads)
    for pairs in (1, 256, 257, most - 1, most):
        for tokens in (0, 16, 8000, 1 << 24, MOST_TOKENS - 16, MOST_TOKENS):
            for cta in (1, 152, 1024):
                _compare(kvrp, pairs, heads, tokens, d, cta, rnd)


def test_refusals(kvrp):  # noqa: F811
    good = dict(pairs=100, heads=4, tokens=8000, head_dim=128, most_cta=152)
    for over in (dict(pairs=-1), dict(pairs=1 << 28), dict(heads=0), dict(heads=4097), dict(tokens=-1), dict(tokens=MOST_TOKENS + 1),
                 dict(head_dim=96), dict(most_cta=0), dict(most_cta=1025), dict(units=[4]), dict(units=[-1]), dict(blocks=[152])):
        a = {**good, **over}
        with pytest.raises(ValueError):
            kvrp.kvrp_test_even_units(a.pop("pairs"), a.pop("heads"), a.pop("tokens"), **a)
