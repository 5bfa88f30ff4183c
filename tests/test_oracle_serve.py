"""Pins of the serving oracle (oracle/serve.py) that need no GPU: e4m3 rounding
against its own code table and torch's cast, the block scale against a search
over exponents, the rotation against the chunk relocation's, growth of an open
block, and attention against the one-query oracle."""
import numpy as np
import pytest
import torch

from oracle import attention, mrope_absolute, rope_absolute
from oracle.serve import E4M3, append_q8, attend_rows, e4m3_round, norm_rows, q8_scale, rotate_magnitude, rotate_rows


def test_e4m3_table_and_ties():
    assert E4M3[0] == 0 and E4M3[1] == 2.0 ** -9 and E4M3[8] == 2.0 ** -6 and E4M3[126] == 448
    assert np.all(np.diff(E4M3) > 0)
    assert np.array_equal(e4m3_round(E4M3), E4M3) and np.array_equal(e4m3_round(-E4M3), -E4M3)
    mid = (E4M3[:-1] + E4M3[1:]) / 2
    even = np.where(np.arange(126) % 2 == 0, E4M3[:-1], E4M3[1:])
    assert np.array_equal(e4m3_round(mid), even)
    assert np.array_equal(e4m3_round(np.nextafter(mid, 0)), E4M3[:-1])
    assert np.array_equal(e4m3_round(np.nextafter(mid, 999)), E4M3[1:])
    assert np.isnan(e4m3_round([np.inf, -np.inf, np.nan])).all()


def test_e4m3_is_torchs_cast():
    x = np.random.default_rng(1).standard_normal(20000).astype(np.float32) * np.exp2(np.arange(20000) % 22 - 14).astype(np.float32)
    x = np.clip(x, -448, 448)
    assert np.array_equal(e4m3_round(x), torch.from_numpy(x).to(torch.float8_e4m3fn).float().numpy())


@pytest.mark.parametrize("amax", [448.0, 449.0, 447.9, 1.0, 1.75, 1.7500001, 3.5, 2.0 ** -100 * 1.76, 2.0 ** -130, 3e38, 0.0])
def test_block_scale_is_the_least_power_of_two(amax):
    s = q8_scale(np.array([amax, -amax / 3, np.inf, np.nan]))
    want = next(e for e in range(-126, 128) if amax <= 448 * 2.0 ** e)
    assert s == 2.0 ** want


def test_rotation_is_the_absolute_rope():
    rng = np.random.default_rng(2)
    x, pos = rng.standard_normal((3, 2, 128)), np.array([0, 17, 40000])
    y = rotate_rows(x, pos, 1e6)
    for h in range(2):
        assert np.allclose(y[:, h], rope_absolute(x[:, h], pos, 1e6), atol=1e-9)
    p3 = np.array([[5, 1, 9], [7, 2, 8], [3, 40, 77]])
    z = rotate_rows(x, p3, 1e6, (16, 24, 24))
    assert np.allclose(z[:, 0], mrope_absolute(x[:, 0], p3.T, 1e6, (16, 24, 24)), atol=1e-9)
    assert np.all(np.abs(y) <= rotate_magnitude(x, pos, 1e6) * (1 + 1e-12))
    assert np.allclose((norm_rows(x, np.ones(128), 0.0) ** 2).mean(-1), 1.0)


def test_open_block_grows_and_keeps_its_earlier_values():
    rng = np.random.default_rng(3)
    values, scale = np.zeros((2, 16, 1, 64)), np.zeros((2, 1))
    first = rng.standard_normal((5, 1, 64))
    append_q8(values, scale, first, [1], 0)
    s0, before = scale[1, 0], values[1, :5].copy()
    append_q8(values, scale, 0.01 * rng.standard_normal((1, 1, 64)), [1], 5)
    assert scale[1, 0] == s0 and np.array_equal(values[1, :5], before)      # smaller rows: nothing moves
    append_q8(values, scale, 100 * rng.standard_normal((1, 1, 64)), [1], 6)
    assert scale[1, 0] > s0
    big = np.abs(before) * (s0 / scale[1, 0]) >= 2.0 ** -6                   # above the subnormals: a shift
    assert np.array_equal((values[1, :5] * scale[1, 0])[big], (before * s0)[big])
    again = values.copy()
    append_q8(values, scale, first, [0], 0)
    assert np.array_equal(values[1], again[1]) and scale[0, 0] == s0


def test_attention_is_the_one_query_oracle():
    rng = np.random.default_rng(4)
    q, k, v = rng.standard_normal((3, 4, 64)), rng.standard_normal((20, 2, 64)), rng.standard_normal((20, 2, 64))
    out, lse, mag = attend_rows(q, k, v, 2, 0.125)
    for i in range(3):
        t = 18 + i
        want = attention(q[i].reshape(-1), k[:t].reshape(t, -1), v[:t].reshape(t, -1), 4, 2, 64, 0.125).reshape(4, 64)
        assert np.allclose(out[i], want, atol=1e-12)
        assert np.allclose(lse[i, 3], np.log(np.exp(0.125 * k[:t, 1] @ q[i, 3]).sum()))
    assert np.all(np.abs(out) <= mag + 1e-12)
