"""kv_step_tables in two launches over more sequences than a block takes at a time (512): what is carried from one
512 to the next, by the blocks that fill the tables and again by the one that moves the state on.

Compared for equality with the oracle, as in test_gpu_step.py."""
import numpy as np
import pytest
import torch

from oracle import step
from test_gpu_step import Tables, batch, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

LARGE = {
    "prefix": dict(n=1300, shared=110, rows=4, ctx=60), "rows": dict(n=2000, rows=16, ctx=60),
    "prefix_short": dict(n=1300, shared=110, rows=40, ctx=60, short=True), "rows_short": dict(n=1100, rows=50, ctx=40, short=True),
    "exact": dict(n=1025, shared=130, rows=20, spare=0), "whole": dict(n=1024, rows=30, ctx=300),
}


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("name", list(LARGE))
def test_two_launches(name, seed):
    t = Tables(**batch(300 + seed, **LARGE[name]))
    t.call()
    assert t.kvrp.kvrp_last_launch_count() == 2
    want = t.check()
    assert bool(want["status"] & step.NO_PAGES) == name.endswith("short")


@pytest.mark.parametrize("name", ["prefix", "rows_short"])
def test_two_launches_in_place(name):
    """kept_lens, held_out and free_state_out in place, positions and slots left out: the second launch reads what the
    first one read, and writes it."""
    t = Tables(**batch(17, **LARGE[name]))
    t.seq_lens.copy_(t.kept)
    t.kvrp.kv_step_tables(t.seq_lens, t.new, t.seqs, held_pages=t.held, free_pages=t.ring, free_state=t.state, prefix=t.prefix,
                          d_status=t.status)
    assert t.kvrp.kvrp_last_launch_count() == 2
    t.positions, t.slots = (torch.as_tensor(step.step_tables(**t.host)[k]).cuda() for k in ("positions", "slots"))
    t.check(held=t.held, state=t.state)


@pytest.mark.parametrize("seed", range(6))
def test_two_launches_bad_input(seed):
    """Counts, pages, lengths and states out of range leave everybody else's outputs as they should be."""
    n = 1200
    rng = np.random.default_rng(seed)
    a = batch(400 + seed, n=n, shared=[0, 120][seed % 2], rows=20)
    for name, values in (("kept", (-1, 1 << 30, 5, 2 ** 31 - 1)), ("new", (-7,)), ("held", (-1, 1, 99999))):
        x = np.array(a[name])
        for v in values:
            x[rng.integers(0, n)] = v
        a[name] = x
    a["new"][n - 100] = 2 ** 31 - 1       # rows past the batch's for all behind it
    table, ring = np.array(a["table"]), np.array(a["ring"])
    table[rng.integers(0, n, 5), rng.integers(0, table.shape[1], 5)] = [-3, len(ring), 2 ** 31 - 1, -2 ** 31, len(ring) + 1]
    ring[rng.integers(0, len(ring), 3)] = [-5, len(ring), 12345678]
    a.update(table=table, ring=ring, n_rows=int(np.clip(a["new"], 0, 20).sum()) + 9)
    if seed == 2:
        a["state"] = [len(ring), 1]
    if seed == 3:
        a["state"] = [a["state"][0], len(ring) + 1]
    if seed == 4:
        a["state"] = [-1, 2]
    if seed == 5:
        a["prefix_len"] = 16 * (len(a["prefix_table"]) + 1)
    t = Tables(**a)
    t.call()
    assert t.kvrp.kvrp_last_launch_count() == 2
    assert t.check()["status"] & step.BAD_LENGTH


def test_many_pages_come_back():
    """Two thirds of 900 sequences end in a step of few rows (one launch) and in one of many (two)."""
    for rows, launches in ((2, 1), (120, 2)):
        a = batch(5, n=900, ctx=800, rows=rows)
        ends = np.arange(900) % 3 > 0
        a["kept"], a["new"] = np.where(ends, 0, a["kept"]), np.where(ends, 0, a["new"])
        t = Tables(**a)
        t.call()
        assert t.kvrp.kvrp_last_launch_count() == launches
        t.check()
