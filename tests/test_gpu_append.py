"""kv_append, kv_append_q8 and kv_pack_q8 against the fp64 oracle (oracle/serve.py).

Bars, derived from the roundings.  Before the store a value is an fp32 evaluation
of y = a cos + b sin with a, b the normed inputs: the mean of d <= 128 squares
(128 2^-24, halved by the square root), rsqrt, weights, the angle (2^-24 of half a
turn) and the products stay below 2^-16 of S = |a cos| + |b sin|.  The store adds
half a step: 2^-8 |y| in bf16; 2^-4 |y| in e4m3, or half its smallest step, 2^-10 of
the block's scale.  Scales are equal unless the largest value lies within 2^-16 of
the border of two of them."""
import numpy as np
import pytest
import torch

from oracle.serve import append_q8, e4m3_round, norm_rows, q8_scale, rotate_magnitude, rotate_rows
from serve_util import bf16, bf16_bits_to_f64, dev, f64, i32, layout

pytestmark = pytest.mark.gpu
F32 = 2.0 ** -16


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()


CASES = {
    "decode": dict(ctx=[0, 1, 14, 15, 16, 31, 500], rows=[1] * 7, hq=28, hkv=4, d=128),
    "decode_64": dict(ctx=[3, 40], rows=[1, 1], hq=8, hkv=8, d=64, norm=True),
    "one_head": dict(ctx=[17], rows=[2], hq=1, hkv=1, d=64),
    "ragged": dict(ctx=[0, 5, 16, 33, 100], rows=[37, 0, 16, 15, 1], hq=14, hkv=2, d=128, norm=True),
    "mrope": dict(ctx=[9, 250], rows=[50, 7], hq=4, hkv=4, d=128, mrope=(16, 24, 24)),
    "wide_group": dict(ctx=[2, 30], rows=[3, 20], hq=48, hkv=3, d=64, norm=True, mrope=(8, 12, 12)),
}


class Batch:
    """One case's inputs, drawn once, and the fp64 rows before any store."""

    def __init__(self, ctx, rows, hq, hkv, d, norm=False, mrope=None, seed=11, theta=1e6, far=0):
        import position_invariant_kv_gb300 as kvrp
        rng = np.random.default_rng(seed)
        self.ctx, self.rows, self.hq, self.hkv, self.d = ctx, rows, hq, hkv, d
        self.lens, self.starts, self.table, self.pages = layout(rng, ctx, rows)
        n = sum(rows)
        size = np.exp(0.5 * rng.standard_normal((hq + 2 * hkv, d)))
        self.qkv = bf16(rng, (n, hq + 2 * hkv, d), size)
        x = bf16_bits_to_f64(self.qkv)
        self.w = [bf16(rng, d, 0.2), bf16(rng, d, 0.2)] if norm else [None, None]
        pos = np.concatenate([np.arange(a, a + b) for a, b in zip(ctx, rows)] + [np.zeros(0, int)]).astype(np.int64)
        self.positions = None
        if mrope:
            pos = np.stack([pos + far, pos // 3, pos % 7 - 3])
            self.positions = pos
        elif far:
            pos = pos + far
            self.positions = pos
        wf = [None if w is None else bf16_bits_to_f64(w) for w in self.w]
        a = [norm_rows(x[:, :hq], wf[0], 1e-5), norm_rows(x[:, hq:hq + hkv], wf[1], 1e-5)]
        self.q, self.k = (rotate_rows(y, pos, theta, mrope) for y in a)
        self.q_mag, self.k_mag = (rotate_magnitude(y, pos, theta, mrope) for y in a)
        self.v = x[:, hq + hkv:]
        self.rng, self.kvrp = rng, kvrp
        self.seqs = kvrp.Seqs(seq_lens=i32(self.lens), block_tables=i32(self.table), num_pages=self.pages, n_rows=n,
                              row_start=i32(self.starts))
        self.dqkv = dev(self.qkv)
        width = (hq + 2 * hkv) * d
        self.q_out = torch.full((n, hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
        self.status = i32([0])
        self.args = dict(n_q_heads=hq, n_kv_heads=hkv, head_dim=d, rope_theta=theta, q_out=self.q_out, q_stride=width,
                         k_stride=width, v_stride=width, norm_eps=1e-5, q_norm=None if not norm else dev(self.w[0]),
                         k_norm=None if not norm else dev(self.w[1]),
                         positions=None if self.positions is None else i32(self.positions), mrope_section=mrope,
                         d_status=self.status)
        self.inputs = (self.dqkv[:, :hq], self.dqkv[:, hq:hq + hkv], self.dqkv[:, hq + hkv:])

    def places(self):
        """(page, slot) of every new row."""
        for s, (a, b) in enumerate(zip(self.ctx, self.rows)):
            for i in range(b):
                yield self.table[s][(a + i) // 16], (a + i) % 16

    def check_q(self):
        assert np.all(np.abs(f64(self.q_out) - self.q) <= 2.0 ** -8 * np.abs(self.q) + F32 * self.q_mag)

    def q8_state(self):
        """An 8-bit cache as earlier calls left it: values and scales (fp64), and on the device."""
        vals, scales = [], []
        for _ in range(2):
            x = self.rng.standard_normal((self.pages, 16, self.hkv, self.d)) * np.exp2(self.rng.integers(-6, 7, (self.pages, 1, self.hkv, 1)))
            s = np.array([[q8_scale(x[p, :, h]) for h in range(self.hkv)] for p in range(self.pages)])
            vals.append(e4m3_round(x / s[:, None, :, None]))
            scales.append(s)
        pool = [torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).cuda() for v in vals]
        return vals, scales, pool, [torch.from_numpy(s.astype(np.float32)).cuda() for s in scales]


@pytest.mark.parametrize("name", CASES)
def test_append_bf16(name):
    b = Batch(**CASES[name])
    pool = [torch.full((b.pages, 16, b.hkv, b.d), float("nan"), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    b.kvrp.kv_append(*b.inputs, b.seqs, k_pool=pool[0], v_pool=pool[1], **b.args)
    assert b.kvrp.kvrp_last_launch_count() == 1
    torch.cuda.synchronize()
    assert int(b.status) == 0
    b.check_q()
    k, v = f64(pool[0]), f64(pool[1])
    seen = np.zeros((b.pages, 16), bool)
    for r, (page, slot) in enumerate(b.places()):
        seen[page, slot] = True
        assert np.all(np.abs(k[page, slot] - b.k[r]) <= 2.0 ** -8 * np.abs(b.k[r]) + F32 * b.k_mag[r])
        assert np.array_equal(v[page, slot], b.v[r])
    assert np.isnan(k[~seen]).all() and np.isnan(v[~seen]).all()      # nothing else was written


def _check_q8(b, got, scale, want, want_scale, mags):
    for pool, sc, w, ws, mag in zip(got, scale, want, want_scale, mags):
        g, gs = f64(pool), f64(sc)
        assert np.array_equal(gs, ws)
        new = np.zeros((b.pages, 16), bool)
        for r, (page, slot) in enumerate(b.places()):
            new[page, slot] = True
            s = ws[page][:, None]
            y = (b.k if mag is not None else b.v)[r]
            room = 2.0 ** -4 * np.abs(y) + 2.0 ** -10 * s + (0 if mag is None else F32 * mag[r])
            assert np.all(np.abs(g[page, slot] * s - y) <= room)
        assert np.array_equal(g[~new], w[~new])      # earlier rows (under the new scale) and untouched slots


@pytest.mark.parametrize("name", CASES)
def test_append_q8(name):
    b = Batch(**CASES[name])
    vals, scales, pool, sc = b.q8_state()
    want, want_scale = [v.copy() for v in vals], [s.copy() for s in scales]
    for j, x in enumerate((b.k, b.v)):
        for s, (a, n) in enumerate(zip(b.ctx, b.rows)):
            append_q8(want[j], want_scale[j], x[b.starts[s]:b.starts[s] + n], b.table[s], a)
    for again in range(2):       # a second call with the same rows changes nothing
        b.kvrp.kv_append_q8(*b.inputs, b.seqs, k_pool=pool[0], v_pool=pool[1], k_scale=sc[0], v_scale=sc[1], **b.args)
        torch.cuda.synchronize()
        assert int(b.status) == 0
        _check_q8(b, pool, sc, want, want_scale, (b.k_mag, None))
    b.check_q()


@pytest.mark.parametrize("far", [2 ** 20 + 12345, 2 ** 31 - 60, -40000])
def test_far_and_negative_positions(far):
    """The angle mod 2 pi holds over the int32 range.  The oracle's fp64 product is itself
    off by up to |position| 2^-53 rad, far below the bar."""
    b = Batch(ctx=[0], rows=[40], hq=2, hkv=2, d=128, far=far)
    pool = [torch.zeros((b.pages, 16, b.hkv, b.d), dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    b.kvrp.kv_append(*b.inputs, b.seqs, k_pool=pool[0], v_pool=pool[1], **b.args)
    torch.cuda.synchronize()
    b.check_q()


def test_token_by_token_is_the_prompt_at_once():
    """bf16: the same bits.  8 bits: the same scales, and values within both stores' half steps."""
    b = Batch(ctx=[0], rows=[40], hq=4, hkv=2, d=64, norm=True)
    shape = (b.pages, 16, b.hkv, b.d)
    one = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    many = [torch.zeros_like(p) for p in one]
    q8 = [[torch.zeros(shape, dtype=torch.uint8, device="cuda") for _ in range(2)] for _ in range(2)]
    sc = [[torch.zeros((b.pages, b.hkv), device="cuda") for _ in range(2)] for _ in range(2)]
    b.kvrp.kv_append(*b.inputs, b.seqs, k_pool=many[0], v_pool=many[1], **b.args)
    b.kvrp.kv_append_q8(*b.inputs, b.seqs, k_pool=q8[0][0], v_pool=q8[0][1], k_scale=sc[0][0], v_scale=sc[0][1], **b.args)
    q_many = b.q_out.clone()
    for i in range(40):
        seqs = b.kvrp.Seqs(seq_lens=i32([i + 1]), block_tables=i32(b.table), num_pages=b.pages)
        x = [t[i:] for t in b.inputs]
        args = dict(b.args, q_out=b.q_out[i:])
        b.kvrp.kv_append(*x, seqs, k_pool=one[0], v_pool=one[1], **args)
        b.kvrp.kv_append_q8(*x, seqs, k_pool=q8[1][0], v_pool=q8[1][1], k_scale=sc[1][0], v_scale=sc[1][1], **args)
    torch.cuda.synchronize()
    assert torch.equal(one[0], many[0]) and torch.equal(one[1], many[1]) and torch.equal(b.q_out, q_many)
    for j in range(2):
        assert torch.equal(sc[0][j], sc[1][j])
        s = f64(sc[0][j])[:, None, :, None]
        a, c = (f64(q8[i][j].view(torch.float8_e4m3fn)) * s for i in range(2))
        assert np.all(np.abs(a - c) <= 2 * (2.0 ** -4 * np.abs(a) + 2.0 ** -10 * s))


def test_values_that_are_not_finite_and_tiny_ones():
    import position_invariant_kv_gb300 as kvrp
    d, hkv = 64, 2
    rng = np.random.default_rng(5)
    v = bf16(rng, (16, hkv, d))
    v[3, 0, 5], v[4, 0, 6] = 0x7F80, 0x7FC0            # inf, NaN
    v[:, 1] = bf16(rng, (16, d), 2.0 ** -120)          # scale floor 2^-126
    v[0, 1, :8] = 0x8000                               # -0
    k = np.zeros_like(v)                               # an all-zero block
    pool = [torch.zeros((1, 16, hkv, d), dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.zeros((1, hkv), device="cuda") for _ in range(2)]
    seqs = kvrp.Seqs(seq_lens=i32([16]), block_tables=i32([[0]]), num_pages=1, n_rows=16, row_start=i32([0, 16]))
    kvrp.kv_append_q8(None, dev(k), dev(v), seqs, n_q_heads=2, n_kv_heads=hkv, head_dim=d, rope_theta=1e4,
                      k_pool=pool[0], v_pool=pool[1], k_scale=sc[0], v_scale=sc[1])
    packed = [torch.zeros_like(pool[0]) for _ in range(2)]
    psc = [torch.zeros_like(sc[0]) for _ in range(2)]
    kvrp.kv_pack_q8(dev(k), dev(v), n_layers=1, n_tokens=16, n_kv_heads=hkv, head_dim=d, k_pool=packed[0], v_pool=packed[1],
                    k_scale=psc[0], v_scale=psc[1], num_pages=1)
    torch.cuda.synchronize()
    x = bf16_bits_to_f64(v)
    want = np.array([q8_scale(x[:, h]) for h in range(hkv)])
    assert np.array_equal(f64(sc[1])[0], want) and np.array_equal(f64(sc[0]), np.full((1, hkv), 2.0 ** -126))
    got = f64(pool[1].view(torch.float8_e4m3fn))[0]
    assert np.array_equal(got, e4m3_round(x / want[None, :, None]), equal_nan=True)
    assert np.isnan(got[3, 0, 5]) and np.isnan(got[4, 0, 6]) and np.isnan(got).sum() == 2
    assert torch.equal(pool[1], packed[1]) and torch.equal(sc[0], psc[0]) and torch.equal(sc[1], psc[1])
    assert np.array_equal(f64(pool[0].view(torch.float8_e4m3fn)), f64(packed[0].view(torch.float8_e4m3fn)))   # a turned 0 may be -0


@pytest.mark.parametrize("layers,tokens,hkv,d,paged", [(1, 1, 1, 64, False), (3, 777, 8, 64, True), (2, 4096, 4, 128, True),
                                                       (2, 33, 3, 128, False), (1, 16, 32, 128, True)])
def test_pack_q8(layers, tokens, hkv, d, paged):
    import position_invariant_kv_gb300 as kvrp
    rng = np.random.default_rng(tokens)
    pages = -(-tokens // 16)
    total = pages + 2
    D = hkv * d
    x = [bf16(rng, (layers, tokens, hkv, d), np.exp2(rng.integers(-20, 20, (layers, tokens, hkv, 1)))) for _ in range(2)]
    table, src_table = rng.permutation(total)[:pages], rng.permutation(total)[:pages]
    src = []
    for y in x:
        if not paged:
            src.append(dev(y))
            continue
        p = np.full((layers, total, 16, hkv, d), 0x7FC0, np.uint16)       # unused slots NaN: they must not count
        for t in range(tokens):
            p[:, src_table[t // 16], t % 16] = y[:, t]
        src.append(dev(p))
    pool = [torch.full((layers, total, 16, hkv, d), 0x55, dtype=torch.uint8, device="cuda") for _ in range(2)]
    sc = [torch.full((layers, total, hkv), -1.0, device="cuda") for _ in range(2)]
    extra = dict(src_table=i32(src_table), src_pages=total) if paged else {}
    status = i32([0])
    kvrp.kv_pack_q8(src[0], src[1], n_layers=layers, n_tokens=tokens, n_kv_heads=hkv, head_dim=d, k_pool=pool[0],
                    v_pool=pool[1], k_scale=sc[0], v_scale=sc[1], block_table=i32(table), num_pages=total, d_status=status,
                    **extra)
    torch.cuda.synchronize()
    assert int(status) == 0
    for y, p, s in zip(x, pool, sc):
        y = np.concatenate([bf16_bits_to_f64(y), np.zeros((layers, pages * 16 - tokens, hkv, d))], 1).reshape(layers, pages, 16, hkv, d)
        amax = np.abs(y).max((2, 4))
        want = np.exp2(np.maximum(-126, np.ceil(np.log2(np.where(amax > 0, amax, 1) / 448))))
        want[0, 0, 0] = q8_scale(y[0, 0, :, 0])
        gs, g = f64(s), f64(p.view(torch.float8_e4m3fn))
        assert np.array_equal(gs[:, table], want)
        assert np.array_equal(g[:, table], e4m3_round(y / want[:, :, None, :, None]))
        rest = np.setdiff1d(np.arange(total), table)
        assert np.all(gs[:, rest] == -1) and bool((p[:, torch.from_numpy(rest)] == 0x55).all())
    assert D * 16 == pool[0][0, 0].numel()


def test_idle_places_bad_lengths_and_bad_pages():
    """An idle sequence (length 0) is skipped without a flag; a length below the rows or past
    the table is flagged and skipped; a bad page is flagged and left out, its q is written."""
    b = Batch(ctx=[3, 20, 40, 7], rows=[1] * 4, hq=4, hkv=2, d=64)
    for lens, table_edit, flags, skipped in (([4, 0, 41, 8], None, 0, [1]), ([4, -2, 41, 8], None, 4, [1]),
                                             ([4, 21, 41, 16 * b.table.shape[1] + 1], None, 4, [3]),
                                             ([4, 2 ** 31 - 1, 41, 8], None, 4, [1]),
                                             (b.lens, (2, 2, b.pages), 1, [2]), (b.lens, (0, 0, -5), 1, [0])):
        table = b.table.copy()
        if table_edit:
            table[table_edit[0], table_edit[1]] = table_edit[2]
        seqs = b.kvrp.Seqs(seq_lens=i32(lens), block_tables=i32(table), num_pages=b.pages)
        pool = [torch.full((b.pages, 16, b.hkv, b.d), 7.0, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
        b.q_out.fill_(9.0)
        b.status.zero_()
        b.kvrp.kv_append(*b.inputs, seqs, k_pool=pool[0], v_pool=pool[1], **b.args)
        torch.cuda.synchronize()
        assert int(b.status) == flags
        for s, (page, slot) in enumerate(b.places()):
            left = bool((pool[1][page, slot] == 7.0).all())
            assert left == (s in skipped)
            assert bool((b.q_out[s] == 9.0).all()) == (s in skipped and table_edit is None)
    # rows out of order or range, ragged form
    for starts in ([0, 2, 1, 3, 4], [0, 1, 2, 3, 9], [-1, 1, 2, 3, 4]):
        seqs = b.kvrp.Seqs(seq_lens=i32(b.lens), block_tables=i32(b.table), num_pages=b.pages, n_rows=4, row_start=i32(starts))
        b.status.zero_()
        b.kvrp.kv_append(*b.inputs, seqs, k_pool=pool[0], v_pool=pool[1], **b.args)
        torch.cuda.synchronize()
        assert int(b.status) == 4


def test_other_stream_and_graph_replay():
    """On a stream of its own, and captured once, replayed as lengths advance on the device."""
    b = Batch(ctx=[0], rows=[20], hq=4, hkv=2, d=128)
    shape = (b.pages, 16, b.hkv, b.d)
    want = [torch.zeros(shape, dtype=torch.bfloat16, device="cuda") for _ in range(2)]
    got = [torch.zeros_like(w) for w in want]
    b.kvrp.kv_append(*b.inputs, b.seqs, k_pool=want[0], v_pool=want[1], **b.args)
    torch.cuda.synchronize()
    lens = i32([1])
    x = b.dqkv[:1].clone()
    seqs = b.kvrp.Seqs(seq_lens=lens, block_tables=i32(b.table), num_pages=b.pages)
    args = dict(b.args, q_out=torch.empty((1, b.hq, b.d), dtype=torch.bfloat16, device="cuda"))
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        b.kvrp.kv_append(x[:, :b.hq], x[:, b.hq:b.hq + b.hkv], x[:, b.hq + b.hkv:], seqs, k_pool=got[0], v_pool=got[1], **args)
    with torch.cuda.stream(side):
        for i in range(20):
            x.copy_(b.dqkv[i:i + 1])
            lens.fill_(i + 1)
            graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
