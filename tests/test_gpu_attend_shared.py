"""kv_attend_shared_q8 against the fp64 oracle (oracle/serve.py), element by element.

The bars are those of kv_attend_q8 (see test_gpu_attend_q8.py): scores, weights and sums are
formed by the same kernels, and what the join adds is fp32: a weight 2^(m - max) of each of the
two passes' parts, off by 2^-21 of itself, and sums of at most a few hundred parts, which the
margin between 2^-11 and 2^-10 covers many times over."""
import numpy as np
import pytest
import torch

from oracle.serve import attend_rows
from serve_util import bf16_bits_to_f64, dev, f64, i32, round_to_bf16_bits
from test_gpu_attend_q8 import Case
from test_gpu_attend_q8_edges import FLOOR, check, send

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()


@pytest.fixture(params=["shared", "each"], autouse=True)
def way(request):
    """The shared tokens read once for the batch, or by each sequence (with few rows), whatever their number."""
    import position_invariant_kv_gb300 as kvrp
    kvrp.kvrp_test_set_each_limit(0 if request.param == "shared" else 1 << 50)
    yield request.param
    kvrp.kvrp_test_set_each_limit(-1)


class Shared(Case):
    """Case with the first `prefix` tokens of all sequences on the same pages, `ctx` own tokens behind
    them; the sequences' own table entries for these pages are -1."""

    def __init__(self, prefix, ctx, rows, hq, hkv, d, over=0, **more):
        super().__init__([prefix + c for c in ctx], rows, hq, hkv, d, **more)
        self.first = prefix // 16
        self.prefix_pages = self.table[0][:self.first].copy()
        self.table[:, :self.first] = self.prefix_pages
        send(self)
        table = self.table.copy()
        table[:, :self.first] = -1
        lens = [0 if s in self.idle else n for s, n in enumerate(self.lens)]
        n = sum(rows)
        self.seqs = self.kvrp.Seqs(seq_lens=i32(lens), block_tables=i32(table), num_pages=self.pages, n_rows=n,
                                   row_start=None if self.one_each else i32(self.starts), max_rows=self.max_rows)
        self.prefix = self.kvrp.Prefix(i32(np.concatenate([self.prefix_pages, [-7]])), i32([prefix + over]))
        most = self.max_rows or n
        self.ws = torch.full((self.kvrp.kv_attend_shared_q8_workspace_size(hq, hkv, d, max(1, most), n),), 0xFF,
                             dtype=torch.uint8, device="cuda")

    def run(self, **over):
        args = dict(n_q_heads=self.hq, n_kv_heads=self.hkv, head_dim=self.d, softmax_scale=self.sm, k_pool=self.pool[0],
                    v_pool=self.pool[1], k_scale=self.dsc[0], v_scale=self.dsc[1], out=self.out, lse=self.lse, workspace=self.ws,
                    d_status=self.status)
        args.update(over)
        q, seqs, prefix = args.pop("q", self.dq), args.pop("seqs", self.seqs), args.pop("prefix", self.prefix)
        self.kvrp.kv_attend_shared_q8(q, seqs, prefix, **args)


FEW = {
    "small": dict(prefix=48, ctx=[0, 1, 14, 15, 16, 30], rows=[1] * 6, hq=28, hkv=4, d=128, one_each=True),
    "one_page": dict(prefix=16, ctx=[0, 3], rows=[1, 1], hq=8, hkv=2, d=64, one_each=True),
    "alone": dict(prefix=320, ctx=[700], rows=[1], hq=7, hkv=1, d=128, one_each=True),
    "no_prefix": dict(prefix=0, ctx=[0, 33, 200], rows=[1] * 3, hq=8, hkv=2, d=128, one_each=True),
    "open_page": dict(prefix=64, over=15, ctx=[20, 16, 40], rows=[1] * 3, hq=8, hkv=2, d=128, one_each=True),
    "long": dict(prefix=6000, ctx=[5, 700, 90], rows=[1] * 3, hq=14, hkv=2, d=128, one_each=True),
    "long_64": dict(prefix=5008, ctx=[5, 700, 90], rows=[1] * 3, hq=8, hkv=2, d=64, one_each=True),
    "group_16": dict(prefix=208, ctx=[40, 100], rows=[1, 1], hq=32, hkv=2, d=128, one_each=True),
    "heads": dict(prefix=96, ctx=[9, 0, 40], rows=[1] * 3, hq=32, hkv=32, d=128, one_each=True),
    "heads_64": dict(prefix=144, ctx=[9, 0, 40], rows=[1] * 3, hq=24, hkv=24, d=64, one_each=True),
    "odd_heads": dict(prefix=256, ctx=[3, 70], rows=[1, 1], hq=21, hkv=3, d=128, one_each=True),
    "batch": dict(prefix=176, ctx=[int(11 * i % 70) for i in range(150)], rows=[1] * 150, hq=4, hkv=2, d=64, one_each=True),
    "row_tiles": dict(prefix=32, ctx=[int(11 * i % 30) for i in range(300)], rows=[1] * 300, hq=8, hkv=8, d=64, one_each=True),
    "drafts": dict(prefix=304, ctx=[0, 13, 31, 150], rows=[4, 3, 2, 4], hq=8, hkv=4, d=64),
    "drafts_128": dict(prefix=1600, ctx=[14, 60, 0], rows=[2, 1, 0], hq=14, hkv=2, d=128),
    "any_scale": dict(prefix=128, ctx=[100, 33], rows=[1, 1], hq=8, hkv=2, d=128, one_each=True, pow2=False),
    "wide_value_scales": dict(prefix=400, ctx=[300, 10], rows=[1, 1], hq=8, hkv=2, d=128, one_each=True, v_spread=30),
    "shares": dict(prefix=15008, ctx=[3, 40], rows=[1, 1], hq=21, hkv=3, d=128, one_each=True),
    "shares_64": dict(prefix=9008, ctx=[5, 40], rows=[2, 1], hq=16, hkv=8, d=64),
    "idle": dict(prefix=80, ctx=[10, 20, 30], rows=[1] * 3, hq=8, hkv=2, d=128, one_each=True, idle=(1,)),
    "all_idle": dict(prefix=80, ctx=[10, 20], rows=[1, 1], hq=8, hkv=2, d=64, one_each=True, idle=(0, 1)),
}
MANY = {
    "two_runs": dict(prefix=304, ctx=[0, 13, 31, 150], rows=[5, 3, 8, 1], hq=8, hkv=2, d=64),
    "three_runs": dict(prefix=160, ctx=[0, 13, 31, 150, 14], rows=[5, 0, 6, 3, 2], hq=14, hkv=2, d=128),
    "four_runs": dict(prefix=48, ctx=[70, 3, 0], rows=[4, 2, 3], hq=32, hkv=2, d=128),
    "four_runs_g1": dict(prefix=48, ctx=[7, 300, 0], rows=[64, 33, 17], hq=3, hkv=3, d=64),
    "one_tile": dict(prefix=160, ctx=[0], rows=[30], hq=4, hkv=2, d=128),
    "long_drafts": dict(prefix=2000, ctx=[30, 0, 77, 200], rows=[5] * 4, hq=28, hkv=4, d=128),
    "ragged": dict(prefix=96, ctx=[0, 130, 17, 50, 3], rows=[37, 1, 0, 64, 129], hq=14, hkv=2, d=128),
    "ragged_64": dict(prefix=512, ctx=[3, 100, 0], rows=[150, 2, 17], hq=8, hkv=4, d=64),
    "units": dict(prefix=16, ctx=[3, 9], rows=[300, 270], hq=16, hkv=16, d=64),
    "more_units_than_sms": dict(prefix=160, ctx=[3, 9], rows=[300, 270], hq=64, hkv=64, d=64),
    "group_16": dict(prefix=64, ctx=[60, 0], rows=[21, 2], hq=32, hkv=2, d=128),
    "no_prefix": dict(prefix=0, ctx=[60, 0], rows=[21, 18], hq=8, hkv=2, d=128),
    "value_scales": dict(prefix=400, ctx=[40], rows=[30], hq=4, hkv=2, d=128, v_spread=30),
    "idle": dict(prefix=32, ctx=[40, 10, 0], rows=[20, 5, 30], hq=4, hkv=4, d=64, idle=(1,)),
    "unspoken_bound": dict(prefix=48, ctx=[9, 8], rows=[19, 14], hq=4, hkv=4, d=128, max_rows=0),
}


@pytest.mark.parametrize("name", [f"few-{n}" for n in FEW] + [f"many-{n}" for n in MANY])
def test_parity(name, way):
    kind, name = name.split("-")
    c = Shared(**(FEW if kind == "few" else MANY)[name])
    c.run()
    runs = -(-(c.max_rows or sum(c.rows)) // (16 // (c.hq // c.hkv)))   # of the rows that the kernel for few takes
    assert c.kvrp.kvrp_last_launch_count() == (2 if way == "each" and runs <= 16 else 3 if runs <= 4 else 4)
    c.check()
    assert int(c.status) == 0
    first = c.out.clone(), c.lse.clone()
    c.out.fill_(3.0)
    c.run()
    torch.cuda.synchronize()
    assert torch.equal(first[0], c.out) and torch.equal(first[1], c.lse)     # the same bits again


@pytest.mark.parametrize("rows", [1, 25])
def test_agrees_with_kv_attend_q8(rows):
    c = Shared(prefix=208, ctx=[90, 5, 300], rows=[rows] * 3, hq=8, hkv=2, d=128)
    c.run()
    both = c.out.clone()
    c.kvrp.kv_attend_q8(c.dq, c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(c.table), num_pages=c.pages, n_rows=3 * rows,
                                          row_start=i32(c.starts), max_rows=rows), n_q_heads=8, n_kv_heads=2, head_dim=128,
                        softmax_scale=c.sm, k_pool=c.pool[0], v_pool=c.pool[1], k_scale=c.dsc[0], v_scale=c.dsc[1], out=c.out,
                        workspace=torch.empty(c.kvrp.kv_attend_q8_workspace_size(8, 2, 128, rows), dtype=torch.uint8, device="cuda"))
    torch.cuda.synchronize()
    a, b = f64(both), f64(c.out)
    for s in range(3):
        x = slice(c.starts[s], c.starts[s + 1])
        _, _, mag = attend_rows(bf16_bits_to_f64(c.q)[x], *c.sequence(s), 2, c.sm)
        assert np.all(np.abs(a[x] - b[x]) <= 2 * (2.0 ** -8 * np.abs(a[x]) + 2.0 ** -10 * mag))


@pytest.mark.parametrize("rows", [[1, 1, 1, 1], [20, 3, 9, 30]])
def test_bad_lengths_leave_their_rows(rows):
    """A sequence that ends inside the prefix, or whose rows begin there, or that is bad by itself."""
    c = Shared(prefix=64, ctx=[20, 30, 5, 40], rows=rows, hq=4, hkv=2, d=64)
    for bad in (64, 63 + rows[1], 3, -1, 16 * c.table.shape[1] + 1):
        lens = list(c.lens)
        lens[1] = bad
        c.out.fill_(5.0)
        c.status.zero_()
        c.run(seqs=c.kvrp.Seqs(seq_lens=i32(lens), block_tables=i32(c.table), num_pages=c.pages, n_rows=sum(rows),
                               row_start=i32(c.starts), max_rows=max(rows)))
        c.check(seqs=[0, 2, 3])
        assert int(c.status) == 4 and bool((c.out[c.starts[1]:c.starts[2]] == 5.0).all()), bad
    if max(rows) > 1:   # more rows than max_rows says
        c.status.zero_()
        c.out.fill_(5.0)
        c.run(seqs=c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(c.table), num_pages=c.pages, n_rows=sum(rows),
                               row_start=i32(c.starts), max_rows=25))
        c.check(seqs=[0, 1, 2])
        assert int(c.status) == 4 and bool((c.out[c.starts[3]:] == 5.0).all())


@pytest.mark.parametrize("rows", [1, 20])
def test_bad_prefix_leaves_all_rows(rows):
    c = Shared(prefix=64, ctx=[20, 30], rows=[rows, rows], hq=4, hkv=2, d=64)
    for length in (-1, 16 * 6, 2 ** 31 - 1, -2 ** 31):
        c.out.fill_(5.0)
        c.status.zero_()
        c.run(prefix=c.kvrp.Prefix(i32(c.prefix_pages), i32([length])))
        torch.cuda.synchronize()
        assert int(c.status) == 4 and bool((c.out == 5.0).all()), length
    for starts in ([0, 3 * rows, 2 * rows], [-1, rows, 2 * rows], [0, rows, 2 * rows + 1], [rows, 0, 2 * rows]):
        c.status.zero_()
        c.run(seqs=c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(c.table), num_pages=c.pages, n_rows=2 * rows,
                               row_start=i32(starts), max_rows=rows))
        torch.cuda.synchronize()
        assert int(c.status) == 4, starts


@pytest.mark.parametrize("rows", [1, 20])
def test_bad_pages_read_as_zeros(rows):
    c = Shared(prefix=64, ctx=[20, 30], rows=[rows, rows], hq=4, hkv=2, d=128)
    for bad in (-1, c.pages, 2 ** 31 - 1):
        pages = c.prefix_pages.copy()
        pages[2] = bad
        keep = [v.copy() for v in c.val]
        for v in c.val:
            v[c.prefix_pages[2]] = 0
        c.status.zero_()
        c.run(prefix=c.kvrp.Prefix(i32(pages), i32([64])))
        c.check()
        assert int(c.status) == 1
        c.val = keep
    table = c.table.copy()
    table[1, 4] = -3                          # its first own page
    c.status.zero_()
    c.run(seqs=c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(table), num_pages=c.pages, n_rows=2 * rows,
                           row_start=i32(c.starts), max_rows=rows))
    c.check(seqs=[0])
    assert int(c.status) == 1


@pytest.mark.parametrize("rows", [1, 20])
def test_part_of_a_batch(rows):
    """Two prefixes: two calls, each over its sequences of the same arrays; other rows stay."""
    a = Shared(prefix=96, ctx=[20, 30, 7, 50], rows=[rows] * 4, hq=8, hkv=2, d=128)
    other = np.array(a.table[3][:6])[::-1].copy()    # sequences 2, 3 begin with these pages instead
    lens, starts, table = i32(a.lens), i32(a.starts), i32(a.table)
    for first, pages in ((0, a.prefix_pages), (2, other)):
        seqs = a.kvrp.Seqs(seq_lens=lens[first:first + 2], block_tables=table[first:first + 2], num_pages=a.pages,
                           n_rows=4 * rows, row_start=starts[first:first + 3], max_rows=rows)
        a.out[2 * rows:].fill_(5.0)
        a.run(seqs=seqs, prefix=a.kvrp.Prefix(i32(pages), i32([96])))
        if first == 0:
            torch.cuda.synchronize()
            assert bool((a.out[2 * rows:] == 5.0).all())
    a.table[2:, :6] = other
    a.check()
    assert int(a.status) == 0


def test_rows_behind_the_last_sequence_stay():
    c = Shared(prefix=96, ctx=[20, 30], rows=[2, 3], hq=8, hkv=2, d=64)
    q = torch.cat([c.dq, torch.full((40, 8, 64), float("nan"), dtype=torch.bfloat16, device="cuda")])
    out = torch.full((45, 8, 64), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((45, 8), 5.0, device="cuda")
    c.ws = torch.empty(c.kvrp.kv_attend_shared_q8_workspace_size(8, 2, 64, 3, 45), dtype=torch.uint8, device="cuda")
    c.run(q=q, out=out, lse=lse, seqs=c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(c.table), num_pages=c.pages, n_rows=45,
                                                  row_start=i32(c.starts), max_rows=3))
    torch.cuda.synchronize()
    assert bool((out[5:] == 5.0).all()) and bool((lse[5:] == 5.0).all())
    c.out, c.lse = out[:5], lse[:5]
    c.check()


@pytest.mark.parametrize("rows", [1, 20])
def test_values_that_are_not_numbers(rows):
    """A NaN value of a shared token reaches all rows, one of an own token its sequence's rows that see it."""
    c = Shared(prefix=48, ctx=[20, 30], rows=[rows, rows], hq=4, hkv=2, d=128)
    pool = c.pool[1].view(torch.uint8)
    page = int(c.prefix_pages[1])
    old = int(pool[page, 5, 1, 9])
    pool[page, 5, 1, 9] = 0x7F
    c.run()
    torch.cuda.synchronize()
    bad = np.isnan(f64(c.out))
    want = np.zeros_like(bad)
    want[:, 2:, 9] = True
    assert np.array_equal(bad, want)
    pool[page, 5, 1, 9] = old
    last = c.lens[1] - 1                     # seen by the last row of sequence 1 alone
    pool[int(c.table[1][last // 16]), last % 16, 0, 3] = 0xFF
    c.run()
    torch.cuda.synchronize()
    bad, want = np.isnan(f64(c.out)), np.zeros_like(bad)
    want[-1, :2, 3] = True
    assert np.array_equal(bad, want)


def test_scores_and_scales_of_the_two_parts_lie_apart():
    """Shared values 2^60 times the own ones and the other way round; one part's scores far above the other's."""
    for part in (0, 1):
        for what in (0, 1):
            c = Shared(prefix=160, ctx=[50, 90], rows=[1, 1], hq=8, hkv=2, d=128)
            pages = c.prefix_pages if part == 0 else np.unique(c.table[:, 10:][c.table[:, 10:] >= 0])
            c.scale[1][pages] *= 2.0 ** (60 if what == 0 else -60)
            if what == 1:
                c.scale[0][pages] *= 2.0 ** -20
            send(c)
            c.run()
            c.check()


def test_projection_rows_and_no_lse():
    c = Shared(prefix=112, ctx=[50, 20], rows=[1, 1], hq=8, hkv=2, d=64, one_each=True)
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


@pytest.mark.parametrize("rows", [1, 20])
def test_graph_replay_follows_lengths_and_prefix(rows):
    c = Shared(prefix=160, ctx=[150, 40], rows=[rows, rows], hq=8, hkv=2, d=128)
    lens, length = i32([160 + rows, 0]), i32([0])
    seqs = c.kvrp.Seqs(seq_lens=lens, block_tables=i32(c.table), num_pages=c.pages, n_rows=2 * rows, row_start=i32(c.starts),
                       max_rows=rows)
    prefix = c.kvrp.Prefix(i32(c.prefix_pages), length)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.run(seqs=seqs, prefix=prefix)
    lens.copy_(i32(c.lens))
    for tokens in (160, 0, 80, 33):
        length.fill_(tokens)
        c.out.fill_(5.0)
        graph.replay()
        c.check()
        assert int(c.status) == 0


def test_two_calls_at_once():
    """Different batches on two streams, a workspace each."""
    cs = [Shared(prefix=p, ctx=[50, 20, 300], rows=[r] * 3, hq=8, hkv=2, d=128, seed=p) for p, r in ((1600, 1), (320, 12))]
    streams = [torch.cuda.Stream() for _ in cs]
    torch.cuda.synchronize()
    for _ in range(10):
        for c, st in zip(cs, streams):
            with torch.cuda.stream(st):
                c.run()
    for c in cs:
        c.check()


@pytest.mark.parametrize("case", [dict(prefix=3200, ctx=[300, 17], rows=[1, 1], hq=14, hkv=2, d=128),
                                  dict(prefix=1600, ctx=[120], rows=[90], hq=8, hkv=2, d=64)])
def test_short_wait_limit_reports_timeout_and_the_next_call_is_right(case, way):
    """The passes' waits give up almost at once; the call returns, says so, and leaves nothing behind."""
    c = Shared(**case)
    if way == "each" and max(c.rows) == 1:
        pytest.skip("no pass with waits")
    if way == "each":
        c.kvrp.kvrp_test_set_each_limit(0)
    try:
        c.kvrp.kvrp_test_set_wait_limit(1)
        c.run()
    finally:
        c.kvrp.kvrp_test_set_wait_limit(0)
    torch.cuda.synchronize()                      # the launches return
    assert int(c.status) & c.kvrp.KVRP_DEV_TIMEOUT
    c.status.zero_()
    c.run()
    c.check()
    assert int(c.status) == 0


SHAPES = {
    "few_128": dict(prefix=320, ctx=[0, 14, 233], rows=[3, 4, 4], hq=4, hkv=2, d=128),
    "few_64": dict(prefix=2000, ctx=[13, 70], rows=[2, 4], hq=16, hkv=4, d=64),
    "many_128": dict(prefix=1600, ctx=[5, 90], rows=[41, 20], hq=7, hkv=1, d=128),
    "many_64": dict(prefix=64, ctx=[0, 150], rows=[70, 30], hq=8, hkv=2, d=64),
}
each_shape = pytest.mark.parametrize("shape", SHAPES)


@each_shape
@pytest.mark.parametrize("size", [-42, -100])
def test_tiny_queries(shape, size):
    """Rows far below one, a row of zeros and one as it was (bars: test_gpu_attend_q8_edges.py)."""
    c = Shared(**SHAPES[shape])
    q = bf16_bits_to_f64(c.q) * np.exp2(size)
    q[0, 0] = 0
    q[-1, -1] /= np.exp2(size)
    c.q = round_to_bf16_bits(q)
    check(c)


@each_shape
def test_queries_of_uneven_elements(shape):
    """Elements of a row up to 2^14 apart, the largest ones few."""
    c = Shared(**SHAPES[shape])
    rng = np.random.default_rng(3)
    c.q = round_to_bf16_bits(bf16_bits_to_f64(c.q) * np.exp2(-rng.integers(0, 15, c.q.shape)))
    check(c)


@each_shape
@pytest.mark.parametrize("where", ["shared", "own", "all"])
def test_zero_values(shape, where):
    """Blocks of zeros, scale 2^-126, in one part or both."""
    c = Shared(**SHAPES[shape])
    for s, n in enumerate(c.lens):
        lo, hi = {"shared": (0, c.first), "own": (c.first, -(-n // 16)), "all": (0, -(-n // 16))}[where]
        c.val[1][c.table[s][lo:hi]], c.scale[1][c.table[s][lo:hi]] = 0, FLOOR
    check(c)
    if where == "all":
        assert bool((c.out == 0).all())


@each_shape
def test_queries_that_are_not_numbers(shape):
    """A row of q with NaN or inf is NaN; the others are what they were."""
    c = Shared(**SHAPES[shape])
    c.run()
    torch.cuda.synchronize()
    want = c.out.clone()
    c.dq = c.dq.clone()
    c.dq[1, 2, 3], c.dq[-1, 0, 5] = float("nan"), float("inf")
    c.run()
    torch.cuda.synchronize()
    bad = torch.zeros(c.out.shape[:2], dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[-1, 0] = True
    assert bool(c.out[bad].isnan().all()) and torch.equal(c.out[~bad], want[~bad])


def test_the_librarys_own_limit():
    """Little that is shared is read by each sequence, much once."""
    import position_invariant_kv_gb300 as kvrp
    kvrp.kvrp_test_set_each_limit(-1)
    for prefix, n, launches in ((160, 3, 2), (3008, 34, 3)):      # 0.5 MB, 105 MB
        c = Shared(prefix=prefix, ctx=[i for i in range(n)], rows=[1] * n, hq=4, hkv=4, d=128, one_each=True)
        c.run()
        assert kvrp.kvrp_last_launch_count() == launches
        c.check(seqs=[0, n - 1])


def test_a_pool_past_32_bits():
    """Pages whose bytes lie past 4 GB of their pools."""
    c = Shared(prefix=48, ctx=[5, 20, 0], rows=[1] * 3, hq=32, hkv=32, d=128, one_each=True)
    pages = 70000
    at, pools, scales = pages - c.pages, [], []
    for pool, scale in zip(c.pool, c.dsc):
        pools.append(torch.empty((pages, *pool.shape[1:]), dtype=torch.uint8, device="cuda"))
        scales.append(torch.empty((pages, scale.shape[1]), device="cuda"))
        pools[-1][at:], scales[-1][at:] = pool, scale
    assert pools[0][at:].data_ptr() - pools[0].data_ptr() > 2 ** 32
    table = np.where(c.table >= 0, c.table + at, -1)
    table[:, :c.first] = -1
    c.run(seqs=c.kvrp.Seqs(seq_lens=i32(c.lens), block_tables=i32(table), num_pages=pages),
          prefix=c.kvrp.Prefix(i32(c.prefix_pages + at), i32([48])), k_pool=pools[0], v_pool=pools[1], k_scale=scales[0],
          v_scale=scales[1])
    c.check()
    assert int(c.status) == 0
