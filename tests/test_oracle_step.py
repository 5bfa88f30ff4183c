"""The oracle of step tables and draft verification against hand values and against the
distribution that verification has to leave."""
import numpy as np
import pytest

from oracle import step


def test_tables_by_hand():
    # 8 pages; the ring holds 5, 6, 7 from place 6 on, past the end of the array
    table = [[0, 1, -1, -1], [2, 3, 4, -1], [-1, -1, -1, -1]]
    got = step.step_tables(kept=[20, 30, 0], new=[13, 1, 3], held=[2, 3, 0], table=table, ring=[7, 9, 9, 9, 9, 9, 5, 6],
                           state=[6, 3], n_rows=20)
    # 33 tokens: 3 pages, one taken (5); 31 tokens: 2 pages, page 4 given back; 3 tokens: one taken (6)
    assert got["table"].tolist() == [[0, 1, 5, -1], [2, 3, 4, -1], [6, -1, -1, -1]]
    assert got["ring"] == [7, 4, 9, 9, 9, 9, 5, 6] and got["state"] == [0, 2]
    assert got["held"] == [3, 2, 1] and got["row_start"] == [0, 13, 14, 17] and got["seq_lens"] == [33, 31, 3]
    assert got["positions"] == list(range(20, 33)) + [30, 0, 1, 2, 0, 0, 0]
    assert got["slots"][:13] == list(range(1 * 16 + 4, 32)) + [5 * 16] and got["slots"][13] == 3 * 16 + 14
    assert got["slots"][14:] == [96, 97, 98, -1, -1, -1] and got["status"] == 0


def test_tables_prefix_and_shortage():
    table = np.full((4, 4), -1)
    got = step.step_tables(kept=[32, 32, 32, 33], new=[5, 16, 17, 1], held=[0, 0, 0, 3], table=table, ring=list(range(10)),
                           state=[9, 2], n_rows=39, prefix_table=[8, 4, 3], prefix_len=47)
    # a page each for the first two; the third asks for two with none left; the fourth asks for none
    assert got["table"].tolist() == [[8, 4, 9, -1], [8, 4, 0, -1], [-1] * 4, [-1] * 4]
    assert got["seq_lens"] == [37, 48, 0, 34] and got["held"] == [3, 3, 0, 3] and got["state"] == [1, 0]
    assert got["status"] == step.NO_PAGES | step.BAD_PAGE   # the fourth's table was never filled
    assert got["slots"][21:38] == [-1] * 17 and got["slots"][38] == -1


def test_tables_pages_that_the_ring_has_no_place_for_are_not_counted():
    # one sequence takes page 6, the other gives 0, 1, 2 back to a ring with two places: 2 is lost, and 6 is not free again
    got = step.step_tables(kept=[0, 0], new=[1, 0], held=[0, 3], table=[[-1] * 3, [0, 1, 2]], ring=[8, 9, 7, 6], state=[3, 2],
                           n_rows=1)
    assert got["table"][0].tolist() == [6, -1, -1] and got["ring"] == [8, 0, 1, 6]
    assert got["state"] == [0, 3] and got["status"] & step.BAD_LENGTH   # free: 8, 0, 1


def test_drawn_token_is_exact_at_the_border():
    p = np.array([[0.25, 0.5, 0.25]], np.float32)
    draw = lambda u: step.verify_sequence(p, None, [0], [0.0], u)[1]  # noqa: E731
    assert draw(0.0) == 0 and draw(0.25 - 2.0 ** -32) == 0 and draw(0.25) == 1
    assert draw(0.75 - 2.0 ** -32) == 1 and draw(0.75) == 2 and draw(1 - 2.0 ** -24) == 2 and draw(1.0) == 2


def test_accept_is_strict():
    p, q = np.array([[0.25, 0.75], [1, 0]], np.float32), np.array([[0.5, 0.5], [0, 0]], np.float32)
    run = lambda u: step.verify_sequence(p, q, [1, 0], [u, 0.0], 0.0)  # noqa: E731
    assert run(0.5)[:2] == (0, 1)                     # 0.5 * 0.5 < 0.25 is false: turned down, 1 has the positive part
    assert run(0.5 - 2.0 ** -24)[:2] == (1, 0)
    none = step.verify_sequence(p, None, [1, 0], [0.25, 0.0], 0.5)
    assert none[:2] == (0, 1)


def test_rows_without_a_positive_part_or_weight():
    same = np.array([[0.5, 0.25], [1, 0]], np.float32)
    assert step.verify_sequence(same, np.ones((2, 2), np.float32), [0, 1], [0.9, 0], 0.7) == (0, 1, False)
    assert step.verify_sequence(np.full((1, 3), np.nan), None, [0], [0], 0.5) == (0, -1, True)
    assert step.verify_sequence(same, same, [0, 7], [0.1, 0], 0.0) == (0, 0, True)


@pytest.mark.parametrize("certain", [False, True])
def test_tokens_follow_the_target(certain):
    """Summed over a grid of the numbers, the first token's share is the target's (up to the grid)."""
    p, q = np.array([0.1, 0.2, 0.3, 0.4], np.float32), np.array([0.4, 0.3, 0.2, 0.1], np.float32)
    grid, share = (np.arange(24) + 0.5) / 24, np.zeros(4)
    for t in range(4):
        for u in grid:
            for v in grid:
                a, token, _ = step.verify_sequence(np.stack([p, p]), None if certain else np.stack([q, q]), [9, t], [u, 0], v)
                share[t if a else token] += (0.25 if certain else q[t]) / len(grid) ** 2
    assert np.abs(share - p).max() < 0.03
