"""kv_attend_q8 where its caches, queries and scores leave the ordinary: zero and tiny values,
tiny queries, value scales far apart, values that are not finite, scores that rise along the
sequence.  Against the fp64 oracle (oracle/serve.py), element by element, in both kernels.

Bars, derived from the roundings.  A query enters the score product with an error of at most
2^-17 of its row's largest element, a score is an fp32 sum of products: a score is off by
delta = 2^-17 scale max|q| sum|k| + 2^-16 scale sum|q k| at most, its weight by 2 delta of
itself (delta is far below 1), and by 2^-11 more from its f16 rounding, which is at most
2^-32 of the row's largest weight times value scale below f16's normal range (values are at
most 448 scales).  Sums are fp32: 2^-11 covers them and the accumulator's corrections, one for
each of at most 2^9 tiles.  The store adds half a bf16 step.  The log-sum-exp is off by 2 delta
and 2^-12, and 2^-20 of its size."""
import numpy as np
import pytest
import torch

from oracle.serve import attend_rows, e4m3_round
from serve_util import bf16, bf16_bits_to_f64, dev, f64, i32, round_to_bf16_bits
from test_gpu_attend_q8 import Case

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()


FLOOR = 2.0 ** -126   # the scale of a block of zeros
# few rows: one tile of columns, two tiles; many rows: one Q tile, several units and parts of them
SHAPES = {
    "few_128": dict(ctx=[0, 14, 333], rows=[3, 4, 4], hq=4, hkv=2, d=128),
    "few_64": dict(ctx=[13, 700], rows=[2, 4], hq=16, hkv=4, d=64),
    "few_long": dict(ctx=[6001], rows=[2], hq=7, hkv=1, d=128),
    "many_128": dict(ctx=[5, 190], rows=[41, 120], hq=7, hkv=1, d=128),
    "many_64": dict(ctx=[0, 250], rows=[70, 90], hq=8, hkv=2, d=64),
    "many_long": dict(ctx=[6000], rows=[40], hq=7, hkv=1, d=128),
    "many_long_64": dict(ctx=[6007], rows=[40], hq=4, hkv=1, d=64),
}
each_shape = pytest.mark.parametrize("shape", SHAPES)


def send(c):
    """The case's values, scales and queries onto the device (slots no sequence uses stay NaN)."""
    used = np.zeros((c.pages, 16), bool)
    for s, n in enumerate(c.lens):
        used[c.table[s][np.arange(n) // 16], np.arange(n) % 16] = True
    for j in range(2):
        t = torch.from_numpy(c.val[j].astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
        t[torch.from_numpy(~used)] = 0x7F
        c.pool[j].copy_(t)
        c.dsc[j].copy_(torch.from_numpy(c.scale[j].astype(np.float32)))
    c.dq = dev(c.q)


def at(c, s, tokens):
    """(page, slot) arrays of tokens of sequence s."""
    tokens = np.asarray(tokens)
    return c.table[s][tokens // 16], tokens % 16


def check(c):
    send(c)
    c.run()
    torch.cuda.synchronize()
    assert int(c.status) == 0
    got, lse = f64(c.out), f64(c.lse)
    q, g = bf16_bits_to_f64(c.q), c.hq // c.hkv
    for s in range(len(c.rows)):
        a, b = c.starts[s], c.starts[s + 1]
        k, v = c.sequence(s)
        with np.errstate(invalid="ignore"):
            ref, ref_lse, mag = attend_rows(q[a:b], k, v, c.hkv, c.sm)
        n = c.lens[s]
        vs = c.scale[1][c.table[s][np.arange(n) // 16]]
        for i in range(b - a):
            t = c.lens[s] - (b - a) + i + 1
            for j in range(c.hq):
                kk, row = k[:t, j // g], q[a + i, j]
                assert np.array_equal(np.isnan(got[a + i, j]), np.isnan(ref[i, j])), (s, i, j)
                assert np.isnan(lse[a + i, j]) == np.isnan(ref_lse[i, j])
                if np.isnan(ref_lse[i, j]):
                    continue
                delta = c.sm * (2.0 ** -17 * np.abs(row).max() * np.abs(kk).sum(1) + 2.0 ** -16 * np.abs(kk) @ np.abs(row)).max()
                assert delta < 2.0 ** -5
                x = c.sm * (kk @ row)
                tiny = t * 2.0 ** -32 * 448 * np.exp(x - ref_lse[i, j] + np.log(vs[:t, j // g])).max()
                ok = ~np.isnan(ref[i, j])
                room = 2.0 ** -8 * np.abs(ref[i, j]) + (2 * delta + 2.0 ** -10) * mag[i, j] + tiny + 2.0 ** -133
                err = np.abs(got[a + i, j] - ref[i, j])
                assert np.all(err[ok] <= room[ok]), (s, i, j, (err[ok] / room[ok]).max())
                assert abs(lse[a + i, j] - ref_lse[i, j]) <= 2 * delta + 2.0 ** -12 + 2.0 ** -20 * abs(ref_lse[i, j]), (s, i, j)


@each_shape
@pytest.mark.parametrize("where", ["all", "first", "middle"])
def test_zero_values(shape, where):
    """Blocks of zero values, which the library writes with the scale 2^-126: everywhere, in the first
    token tiles, and over the part of a long context at which some CTAs' shares begin."""
    c = Case(**SHAPES[shape])
    for s, n in enumerate(c.lens):
        pages = -(-n // 16)
        lo, hi = {"all": (0, pages), "first": (0, min(pages, 8)), "middle": (pages // 6, 5 * pages // 6)}[where]
        c.val[1][c.table[s][lo:hi]], c.scale[1][c.table[s][lo:hi]] = 0, FLOOR
    check(c)
    if where == "all":
        assert bool((c.out == 0).all())


@each_shape
@pytest.mark.parametrize("size", [-42, -60, -100])
def test_tiny_queries(shape, size):
    """Rows far below one, and a row of zeros: the mean of the values."""
    c = Case(**SHAPES[shape])
    q = bf16_bits_to_f64(c.q) * np.exp2(size)
    q[0, 0] = 0
    q[-1, -1] /= np.exp2(size)
    c.q = round_to_bf16_bits(q)
    check(c)


@each_shape
def test_tiny_softmax_scale(shape):
    c = Case(**SHAPES[shape])
    c.sm = 1e-30
    check(c)


@each_shape
@pytest.mark.parametrize("size", [-30, 116])
def test_keys_at_the_scale_floor(shape, size):
    """Keys in blocks of the smallest scale, under queries for which the scores vanish and under ones so
    large that they do not."""
    c = Case(**SHAPES[shape])
    c.scale[0][:] = FLOOR
    c.q = round_to_bf16_bits(bf16_bits_to_f64(c.q) * np.exp2(size) * (2.0 if size > 0 else 1.0))
    check(c)


@each_shape
@pytest.mark.parametrize("what", ["v", "v_all_heads", "k"])
def test_nan_in_a_later_row(shape, what):
    """A value that is not finite reaches the rows that see its token, no others."""
    c = Case(**SHAPES[shape])
    for s, n in enumerate(c.lens):
        rows = c.rows[s]
        for token, feature in ((n - 1, 3), (n - 1, c.d - 1), (n - rows // 2 - 1, 17), (n - rows // 2 - 1, 3)):
            page, slot = at(c, s, token)
            head = slice(None) if what == "v_all_heads" else c.hkv - 1
            c.val[0 if what == "k" else 1][page, slot, head, feature] = np.nan
    check(c)


@each_shape
@pytest.mark.parametrize("token", [0, 100])
def test_nan_before_all_rows(shape, token):
    c = Case(**SHAPES[shape])
    for s, n in enumerate(c.lens):
        page, slot = at(c, s, min(token, n - 1))
        c.val[1][page, slot, 0, 5] = np.nan
    check(c)


def along(c, s, steps):
    """Keys of sequence s and all queries nearly along one direction: the scores of token t rise by steps[t] (natural units)."""
    rng = np.random.default_rng(3)
    u = np.sign(rng.standard_normal(c.d))
    n = c.lens[s]
    k = np.asarray(steps)[:, None, None] * u * (0.25 / (c.sm * c.d)) + 0.05 * rng.standard_normal((n, c.hkv, c.d))
    page, slot = at(c, s, np.arange(n))
    for p in np.unique(page):
        mine = page == p
        top = np.abs(k[mine]).max((0, 2))
        c.scale[0][p] = np.exp2(np.ceil(np.log2(top / 448)))
    c.val[0][page, slot] = e4m3_round(k / c.scale[0][page][:, :, None])
    a, b = c.starts[s], c.starts[s + 1]
    c.q[a:b] = bf16(rng, (b - a, c.hq, c.d), 0.1)
    c.q[a:b] = round_to_bf16_bits(bf16_bits_to_f64(c.q[a:b]) + 4 * u)


@each_shape
@pytest.mark.parametrize("form", ["rise", "saw", "fall"])
def test_scores_that_rise(shape, form):
    """The running maximum moves many times: the sum and the accumulator are scaled down with it."""
    c = Case(**SHAPES[shape])
    for s, n in enumerate(c.lens):
        t = np.arange(n) / n
        along(c, s, {"rise": 60 * t, "saw": 40 * t + 20 * (np.arange(n) // 16 % 3), "fall": 60 * (1 - t)}[form])
    check(c)


@each_shape
def test_any_value_scales(shape):
    check(Case(**SHAPES[shape], v_spread=30, pow2=False))


@each_shape
@pytest.mark.parametrize("gap", [0, 20, 60])
@pytest.mark.parametrize("low,high", [(-40, 0), (-100, 20)])
def test_weight_on_pages_of_small_value_scales(shape, gap, low, high):
    """Every other run of pages holds values `high - low` octaves larger, under scores `gap` lower."""
    c = Case(**SHAPES[shape])
    for s, n in enumerate(c.lens):
        small = np.arange(n) // 16 % 8 >= 4
        along(c, s, gap * small.astype(float))
        page, _ = at(c, s, np.arange(n))
        c.scale[1][page] *= np.exp2(np.where(small, low, high))[:, None]
    check(c)


@each_shape
def test_tiny_values(shape):
    """Values near fp32's smallest normal numbers."""
    c = Case(**SHAPES[shape])
    c.scale[1][:] = 2.0 ** -125
    check(c)
