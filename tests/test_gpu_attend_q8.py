"""kv_attend_q8 against the fp64 oracle (oracle/serve.py), element by element.

Bars, derived from the roundings.  The cache's values are exact inputs.  A query enters
the score product with an error of at most 2^-18 of its row's largest element (and none
where bf16's 8 bits fit), a score is an fp32 sum of head_dim products: its error is below
2^-16 of scale * sum_i |q_i k_i|, which the cases keep under 16, so 2^-12 absolute.  The
softmax weights are then off by 2^-12 relative, and by 2^-11 from their f16 rounding
(2^-12 half steps counted twice for the value scale's factor); sums are fp32.  Together
below 2^-10 of sum_t p_t |v_t|; the store adds half a bf16 step, 2^-8 |out|.  The
log-sum-exp is fp32: 2^-12 for the scores, 2^-20 of its size."""
import numpy as np
import pytest
import torch

from oracle.serve import attend_rows, e4m3_round, q8_scale
from serve_util import bf16, bf16_bits_to_f64, dev, f64, i32, layout

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()


class Case:
    """A ragged batch over an 8-bit cache; slots no sequence uses hold NaN bytes."""

    def __init__(self, ctx, rows, hq, hkv, d, seed=21, one_each=False, v_spread=3, q_size=0.7, pow2=True, max_rows=None, idle=()):
        import position_invariant_kv_gb300 as kvrp
        rng = np.random.default_rng(seed)
        self.kvrp, self.hq, self.hkv, self.d, self.rows, self.ctx = kvrp, hq, hkv, d, rows, ctx
        self.lens, self.starts, self.table, self.pages = layout(rng, ctx, rows)
        shape = (self.pages, 16, hkv, d)
        self.val, self.scale = [], []
        for spread in (1, v_spread):
            x = rng.standard_normal(shape)
            s = np.array([[q8_scale(x[p, :, h]) for h in range(hkv)] for p in range(self.pages)])
            v = e4m3_round(x / s[:, None, :, None])
            s = s * np.exp2(rng.integers(-spread, spread + 1, s.shape)) if spread > 1 else s
            if not pow2:
                s = (s * rng.uniform(0.6, 1.7, s.shape)).astype(np.float32).astype(np.float64)
            self.val.append(v)
            self.scale.append(s)
        self.q = bf16(rng, (sum(rows), hq, d), q_size * np.exp(0.5 * rng.standard_normal(d)))
        self.sm = d ** -0.5
        self.one_each = one_each
        used = np.zeros((self.pages, 16), bool)
        for s, n in enumerate(self.lens):
            for t in range(n):
                used[self.table[s][t // 16], t % 16] = True
        self.pool = []
        for v in self.val:
            t = torch.from_numpy(v.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)
            t[torch.from_numpy(~used)] = 0x7F                      # NaN
            self.pool.append(t.cuda())
        self.dsc = [torch.from_numpy(s.astype(np.float32)).cuda() for s in self.scale]
        self.dq = dev(self.q)
        lens = list(self.lens)
        for s in idle:
            lens[s] = 0
        self.idle = idle
        n = sum(rows)
        self.max_rows = max(rows) if max_rows is None else max_rows
        self.seqs = kvrp.Seqs(seq_lens=i32(lens), block_tables=i32(self.table), num_pages=self.pages, n_rows=n,
                              row_start=None if one_each else i32(self.starts), max_rows=self.max_rows)
        self.out = torch.full((n, hq, d), 5.0, dtype=torch.bfloat16, device="cuda")
        self.lse = torch.full((n, hq), 5.0, device="cuda")
        self.status = i32([0])
        self.ws = torch.full((kvrp.kv_attend_q8_workspace_size(hq, hkv, d, max(1, self.max_rows)),), 0xFF, dtype=torch.uint8, device="cuda")

    def run(self, **over):
        args = dict(n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=self.d, softmax_scale=self.sm, k_pool=self.pool[0],
                    v_pool=self.pool[1], k_scale=self.dsc[0], v_scale=self.dsc[1], out=self.out, lse=self.lse, workspace=self.ws,
                    d_status=self.status)
        args.update(over)
        q, seqs = args.pop("q", self.dq), args.pop("seqs", self.seqs)
        self.kvrp.kv_attend_q8(q, seqs, **args)

    def sequence(self, s):
        n = self.lens[s]
        t = np.arange(n)
        page = self.table[s][t // 16]
        return [v[page, t % 16] * sc[page][:, :, None] for v, sc in zip(self.val, self.scale)]

    def check(self, seqs=None):
        torch.cuda.synchronize()
        got, lse = f64(self.out), f64(self.lse)
        q = bf16_bits_to_f64(self.q)
        for s in range(len(self.rows)) if seqs is None else seqs:
            a, b = self.starts[s], self.starts[s + 1]
            if s in self.idle:
                assert np.all(got[a:b] == 0) and np.all(np.isneginf(lse[a:b]))
                continue
            if a == b:
                continue
            k, v = self.sequence(s)
            ref, ref_lse, mag = attend_rows(q[a:b], k, v, self.hkv, self.sm)
            big = self.sm * np.abs(q[a:b]).reshape(b - a, self.hkv, -1, self.d) @ np.abs(k).transpose(1, 2, 0)[None]
            assert big.max() < 16
            err = np.abs(got[a:b] - ref)
            assert np.all(err <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag), (s, (err / mag).max())
            assert np.all(np.abs(lse[a:b] - ref_lse) <= 2.0 ** -12 + 2.0 ** -20 * np.abs(ref_lse)), s


DECODE = {
    "short": dict(ctx=[0, 1, 14, 15, 16, 30, 127, 128], rows=[1] * 8, hq=28, hkv=4, d=128, one_each=True),
    "d64": dict(ctx=[0, 5, 200, 333], rows=[1] * 4, hq=8, hkv=8, d=64, one_each=True),
    "group_16": dict(ctx=[40, 700], rows=[1, 1], hq=32, hkv=2, d=128, one_each=True),
    "group_16_d64": dict(ctx=[17, 410], rows=[1, 1], hq=16, hkv=1, d=64, one_each=True),
    "group_9": dict(ctx=[100], rows=[1], hq=27, hkv=3, d=128, one_each=True),
    "long_alone": dict(ctx=[9000], rows=[1], hq=7, hkv=1, d=128, one_each=True),
    "uneven": dict(ctx=[3, 5000, 17, 64, 1200, 0], rows=[1] * 6, hq=4, hkv=2, d=64, one_each=True),
    "verify": dict(ctx=[0, 13, 31, 450], rows=[4, 3, 2, 4], hq=8, hkv=4, d=64),
    "verify_128": dict(ctx=[14, 600, 0], rows=[2, 1, 0], hq=14, hkv=2, d=128),
    "any_scale": dict(ctx=[100, 333], rows=[1, 1], hq=8, hkv=2, d=128, one_each=True, pow2=False),
    "wide_value_scales": dict(ctx=[300], rows=[1], hq=8, hkv=2, d=128, one_each=True, v_spread=30),
    "many": dict(ctx=[int(7 * i % 90) for i in range(300)], rows=[1] * 300, hq=2, hkv=1, d=64, one_each=True),
    "idle": dict(ctx=[10, 20, 30], rows=[1] * 3, hq=8, hkv=2, d=128, one_each=True, idle=(1,)),
    "all_idle": dict(ctx=[10, 20], rows=[1, 1], hq=8, hkv=2, d=64, one_each=True, idle=(0, 1)),
}


@pytest.mark.parametrize("name", DECODE)
def test_few_rows(name):
    c = Case(**DECODE[name])
    c.run()
    assert c.kvrp.kvrp_last_launch_count() == 2
    c.check()
    assert int(c.status) == 0
    first = c.out.clone(), c.lse.clone()
    c.out.fill_(3.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)     # the same bits again


PROMPT = {
    "one_tile": dict(ctx=[0], rows=[30], hq=4, hkv=2, d=128, max_rows=30),
    "one_tile_d64": dict(ctx=[5], rows=[20], hq=2, hkv=2, d=64),
    "two_q_tiles": dict(ctx=[100], rows=[40], hq=7, hkv=1, d=128),
    "ragged": dict(ctx=[0, 130, 17, 500, 3], rows=[37, 1, 0, 64, 129], hq=14, hkv=2, d=128),
    "ragged_d64": dict(ctx=[3, 1000, 0], rows=[150, 2, 17], hq=8, hkv=4, d=64),
    "group_1": dict(ctx=[250], rows=[300], hq=2, hkv=2, d=64),
    "group_16": dict(ctx=[60, 0], rows=[21, 2], hq=32, hkv=2, d=128),
    "long_context": dict(ctx=[6000], rows=[18], hq=7, hkv=1, d=128),
    "any_scale": dict(ctx=[300], rows=[30], hq=4, hkv=2, d=128, pow2=False),
    "value_scales": dict(ctx=[400], rows=[30], hq=4, hkv=2, d=128, v_spread=6),
    "idle": dict(ctx=[40, 10, 0], rows=[20, 5, 30], hq=4, hkv=4, d=64, idle=(1,)),
    "mixed_tiles": dict(ctx=[2500 + 90 * i for i in range(10)], rows=[150, 20, 130, 9, 20, 140, 1, 30, 129, 128], hq=8, hkv=8, d=64),
    "unspoken_bound": dict(ctx=[9, 8], rows=[19, 14], hq=4, hkv=4, d=128, max_rows=0),
}


@pytest.mark.parametrize("name", PROMPT)
def test_many_rows(name):
    c = Case(**PROMPT[name])
    if c.max_rows == 0:
        c.ws = torch.empty(c.kvrp.kv_attend_q8_workspace_size(c.hq, c.hkv, c.d, sum(c.rows)), dtype=torch.uint8, device="cuda")
    c.run()
    assert c.kvrp.kvrp_last_launch_count() == 2
    c.check()
    assert int(c.status) == 0
    first = c.out.clone(), c.lse.clone()
    c.out.fill_(3.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)


def test_a_prompt_is_its_rows_one_by_one():
    """The kernel for many rows against the one for few, on the same cache."""
    c = Case(ctx=[90], rows=[25], hq=8, hkv=2, d=128)
    c.run()
    one = torch.empty_like(c.out)
    for i in range(25):
        seqs = c.kvrp.Seqs(seq_lens=i32([91 + i]), block_tables=i32(c.table), num_pages=c.pages)
        c.run(seqs=seqs, q=c.dq[i:], out=one[i:], lse=None)
    torch.cuda.synchronize()
    _, _, mag = attend_rows(bf16_bits_to_f64(c.q), *c.sequence(0), 2, c.sm)
    a, b = f64(c.out), f64(one)
    assert np.all(np.abs(a - b) <= 2 * (2.0 ** -8 * np.abs(a) + 2.0 ** -10 * mag))


def test_prompt_bad_lengths_and_bad_pages():
    c = Case(ctx=[60, 30, 90], rows=[20, 20, 40], hq=4, hkv=2, d=64)
    for lens in ([80, 19, 130], [80, 16 * c.table.shape[1] + 1, 130]):
        c.out.fill_(5.0)
        c.status.zero_()
        c.run(seqs=c.kvrp.Seqs(seq_lens=i32(lens), block_tables=i32(c.table), num_pages=c.pages, n_rows=80,
                               row_start=i32(c.starts), max_rows=40))
        c.check(seqs=[0, 2])
        assert int(c.status) == 4 and bool((c.out[20:40] == 5.0).all())
    for bad in (-1, c.pages):
        table = c.table.copy()
        table[1, 0] = bad
        c.status.zero_()
        c.run(seqs=c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(table), num_pages=c.pages, n_rows=80,
                               row_start=i32(c.starts), max_rows=40))
        c.check(seqs=[0, 2])
        assert int(c.status) == 1


def test_zero_values_and_zero_queries():
    """A page of zero values beside others (its scale is the floor), and a query of zeros."""
    c = Case(ctx=[100], rows=[1], hq=4, hkv=1, d=128, one_each=True)
    page = c.table[0][2]
    c.val[1][page], c.scale[1][page] = 0, 2.0 ** -126
    c.pool[1][int(page)] = 0
    c.dsc[1][int(page)] = 2.0 ** -126
    c.q[0, 1] = 0
    c.dq = dev(c.q)
    c.run()
    c.check()


def test_rows_of_a_fused_projection_and_no_lse():
    c = Case(ctx=[50, 20], rows=[1, 1], hq=8, hkv=2, d=64, one_each=True)
    wide = torch.zeros((2, 12, 64), dtype=torch.bfloat16, device="cuda")
    wide[:, :8] = c.dq
    c.run()
    torch.cuda.synchronize()
    want = c.out.clone()
    c.out.zero_()
    c.lse.fill_(5.0)
    c.run(q=wide, q_stride=12 * 64, lse=None)
    torch.cuda.synchronize()
    assert torch.equal(c.out, want) and bool((c.lse == 5.0).all())


def test_nan_stays_in_its_sequence_and_head():
    c = Case(ctx=[70, 70], rows=[1, 1], hq=4, hkv=2, d=128, one_each=True)
    c.pool[0].view(torch.uint8)[int(c.table[0][1]), 3, 1, 7] = 0x7F
    c.run()
    c.check(seqs=[1])
    out = f64(c.out)[0]
    assert np.isnan(out[2:]).all() and np.isfinite(out[:2]).all()


def test_bad_lengths_and_bad_pages():
    c = Case(ctx=[60, 30, 90], rows=[1] * 3, hq=4, hkv=2, d=64, one_each=True)
    for lens in ([61, -1, 91], [61, 16 * c.table.shape[1] + 1, 91]):
        c.out.fill_(5.0)
        c.status.zero_()
        c.run(seqs=c.kvrp.Seqs(seq_lens=i32(lens), block_tables=i32(c.table), num_pages=c.pages))
        c.check(seqs=[0, 2])
        assert int(c.status) == 4 and bool((c.out[1] == 5.0).all())
    for bad in (-1, c.pages, 2 ** 31 - 1):
        table = c.table.copy()
        table[1, 0] = bad
        c.status.zero_()
        c.run(seqs=c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(table), num_pages=c.pages))
        c.check(seqs=[0, 2])
        assert int(c.status) == 1
    # more rows than max_rows says
    c = Case(ctx=[60, 30], rows=[2, 4], hq=4, hkv=4, d=64, max_rows=2)
    c.run()
    c.check(seqs=[0])
    assert int(c.status) == 4 and bool((c.out[2:] == 5.0).all())


def test_shared_pages_and_other_stream():
    """Two sequences over one prefix's pages; the call on a stream of its own."""
    c = Case(ctx=[200, 200], rows=[1, 1], hq=8, hkv=2, d=128, one_each=True)
    c.table[1] = c.table[0]
    seqs = c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(c.table), num_pages=c.pages)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        c.run(seqs=seqs)
    c.check()


def test_graph_replay_follows_the_lengths():
    c = Case(ctx=[150, 40], rows=[1, 1], hq=8, hkv=2, d=128, one_each=True)
    lens = i32([100, 41])
    seqs = c.kvrp.Seqs(seq_lens=lens, block_tables=i32(c.table), num_pages=c.pages)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(seqs=seqs)
    lens.copy_(i32(c.lens))
    graph.replay()
    c.check()
