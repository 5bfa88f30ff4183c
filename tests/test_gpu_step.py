"""kv_step_tables and kv_verify_drafts against the oracle (oracle/step.py).

All outputs are whole numbers, so every comparison is for equality: tables, rings, lengths,
positions and slots; tokens, counts and kept lengths."""
import numpy as np
import pytest
import torch

from oracle import step
from serve_util import i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()


# --- step tables -----------------------------------------------------------------------
class Tables:
    """A batch's arrays on the host and on the device, and the call."""

    def __init__(self, kept, new, held, table, ring, state, n_rows=None, prefix_table=None, prefix_len=0):
        import position_invariant_kv_gb300 as kvrp
        self.kvrp = kvrp
        self.host = dict(kept=kept, new=new, held=held, table=np.array(table), ring=list(ring), state=list(state),
                         n_rows=sum(max(0, int(x)) for x in new) if n_rows is None else n_rows)
        if prefix_table is not None:
            self.host.update(prefix_table=prefix_table, prefix_len=prefix_len)
        h = self.host
        self.table, self.ring, self.status = i32(table), i32(ring), i32([0])
        self.kept, self.new, self.held, self.state = i32(kept), i32(new), i32(held), i32(state)
        self.held_out, self.state_out = i32([-9] * len(kept)), i32([-9, -9])
        self.row_start, self.seq_lens = i32([-9] * (len(kept) + 1)), i32([-9] * len(kept))
        self.positions = torch.full((h["n_rows"],), -9, dtype=torch.int32, device="cuda")
        self.slots = torch.full((h["n_rows"],), -9, dtype=torch.int64, device="cuda")
        self.seqs = kvrp.Seqs(seq_lens=self.seq_lens, block_tables=self.table, num_pages=len(ring), n_rows=h["n_rows"],
                              row_start=self.row_start)
        self.prefix = kvrp.Prefix(i32(prefix_table), i32([prefix_len])) if prefix_table is not None else None

    def call(self, **over):
        args = dict(held_pages=self.held, held_out=self.held_out, free_pages=self.ring, free_state=self.state,
                    free_state_out=self.state_out, prefix=self.prefix, positions=self.positions, slots=self.slots,
                    d_status=self.status)
        args.update(over)
        self.kvrp.kv_step_tables(self.kept, self.new, self.seqs, **args)

    def check(self, held=None, state=None, seq_lens=None):
        torch.cuda.synchronize()
        want = step.step_tables(**self.host)
        got = dict(table=self.table, ring=self.ring, held=self.held_out if held is None else held,
                   state=self.state_out if state is None else state, row_start=self.row_start,
                   seq_lens=self.seq_lens if seq_lens is None else seq_lens, positions=self.positions, slots=self.slots)
        for name, t in got.items():
            assert np.array_equal(t.cpu().numpy(), np.array(want[name]).reshape(t.shape)), name
        assert int(self.status) == want["status"]
        return want


def batch(seed, n, ctx=200, rows=6, shared=0, short=False, spare=5):
    """A consistent batch: sequences that go on (some with fewer tokens than they had), begin and end."""
    rng = np.random.default_rng(seed)
    kind = rng.integers(0, 5, n)
    had = rng.integers(0, ctx, n) + 16 * shared
    kept = np.where(kind == 0, 0, np.where(kind == 1, 16 * shared, np.maximum(had - rng.integers(0, 40, n), 16 * shared)))
    new = np.where(kind == 0, 0, rng.integers(0, rows + 1, n))
    held = np.where(kind == 1, 0, -(-had // 16))
    held = np.where((held > 0) & (held < shared), shared, held)
    new = np.where((kept == 0) & (new == 0), 0, new)
    need = -(-(kept + new) // 16)
    lacks = np.where(need > 0, np.maximum(0, need - np.maximum(held, shared)), 0).sum()
    own = np.maximum(held - shared, 0)
    free = int(lacks) // 2 if short else int(lacks) + spare
    size = shared + int(own.sum()) + free
    size = max(size, 1)
    order = rng.permutation(size)
    table = np.full((n, int(max(need.max(), held.max())) + 2), -1)
    at = shared
    for s in range(n):
        if held[s]:
            table[s, :shared] = order[:shared]
            table[s, shared:held[s]] = order[at:at + own[s]]
            at += own[s]
    ring, head = np.full(size, -1), int(rng.integers(0, size))
    ring[(head + np.arange(free)) % size] = order[at:at + free]
    args = dict(kept=kept, new=new, held=held, table=table, ring=ring, state=[head, free])
    if shared:
        args.update(prefix_table=order[:shared], prefix_len=16 * shared + int(rng.integers(0, 16)))
    return args


TABLES = {
    "one": dict(n=1), "few": dict(n=7), "decode": dict(n=64), "block": dict(n=512), "blocks": dict(n=513, rows=3),
    "many": dict(n=3000, rows=4, ctx=60), "prefix": dict(n=40, shared=37), "prompts": dict(n=20, rows=3000),
    "prompts_prefix": dict(n=300, rows=200, shared=70), "short": dict(n=50, rows=60, short=True),
    "short_prefix": dict(n=600, rows=20, shared=3, short=True), "exact": dict(n=30, rows=60, spare=0),
    "no_rows": dict(n=33, rows=0),
}


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("name", list(TABLES))
def test_tables(name, seed):
    t = Tables(**batch(100 + seed, **TABLES[name]))
    t.call()
    want = t.check()
    assert bool(want["status"] & step.NO_PAGES) == (name.startswith("short"))
    launches = t.kvrp.kvrp_last_launch_count()
    assert launches == (2 if name in ("prompts", "prompts_prefix") else 1)


@pytest.mark.parametrize("name", ["few", "blocks", "prompts", "short_prefix"])
def test_tables_in_place_and_without_rows(name):
    """held_out, free_state_out and kept_lens in place; positions and slots left out."""
    t = Tables(**batch(7, **TABLES[name]))
    t.positions, t.slots = t.positions.fill_(0), t.slots.fill_(0)
    t.seq_lens.copy_(t.kept)
    t.kvrp.kv_step_tables(t.seq_lens, t.new, t.seqs, held_pages=t.held, free_pages=t.ring, free_state=t.state, prefix=t.prefix,
                          d_status=t.status)
    torch.cuda.synchronize()
    assert not t.positions.any() and not t.slots.any()
    t.positions, t.slots = (torch.as_tensor(step.step_tables(**t.host)[k]).cuda() for k in ("positions", "slots"))
    t.check(held=t.held, state=t.state)


@pytest.mark.parametrize("seed", range(6))
def test_tables_bad_input(seed):
    """Counts, pages and lengths out of range leave everybody else's outputs as they should be."""
    rng = np.random.default_rng(seed)
    a = batch(200 + seed, n=60, shared=[0, 4][seed % 2], rows=20)
    for name, values in (("kept", (-1, 1 << 30, 5, 2 ** 31 - 1)), ("new", (-7, 1 << 30, 2 ** 31 - 1)), ("held", (-1, 1, 99999))):
        x = np.array(a[name])
        for v in values:
            x[rng.integers(0, 60)] = v
        a[name] = x
    table, ring = np.array(a["table"]), np.array(a["ring"])
    table[rng.integers(0, 60, 5), rng.integers(0, table.shape[1], 5)] = [-3, len(ring), 2 ** 31 - 1, -2 ** 31, len(ring) + 1]
    ring[rng.integers(0, len(ring), 3)] = [-5, len(ring), 12345678]
    a.update(table=table, ring=ring, n_rows=int(np.clip(a["new"], 0, 20).sum()) + 9)
    if seed == 3:
        a["state"] = [a["state"][0], len(ring) + 1]
    if seed == 4:
        a["state"] = [-1, 2]
    if seed == 5:
        a["prefix_len"] = 16 * (len(a["prefix_table"]) + 1)
    t = Tables(**a)
    t.call()
    assert t.check()["status"] & step.BAD_LENGTH


def test_tables_more_back_than_the_ring_holds():
    t = Tables(kept=[0, 0], new=[0, 0], held=[3, 3], table=[[0, 1, 2], [0, 1, 3]], ring=[9, 9, 9, 9], state=[3, 2])
    t.call()
    assert t.check()["status"] == step.BAD_LENGTH


@pytest.mark.parametrize("behind", [0, 9000])   # rows behind the last sequence: one launch, two
def test_tables_take_and_lose_pages_in_one_call(behind):
    """Pages that are lost are not counted: no page of a served table is among the free ones afterwards."""
    size, n = 40, 6
    table = np.full((n, 12), -1)
    for s, pages in ((1, range(0, 12)), (3, range(12, 24)), (5, range(24, 27))):
        table[s, :len(pages)] = list(pages)
    ring = [(x + 27) % size for x in range(size)]       # free: 27 to 39, and of the ended ones' pages what the books say wrongly
    t = Tables(kept=[0, 0, 0, 0, 0, 48], new=[33, 0, 17, 0, 3, 2], held=[0, 12, 0, 12, 0, 3], table=table, ring=ring, state=[5, 30],
               n_rows=55 + behind)
    t.call()
    want = t.check()
    assert t.kvrp.kvrp_last_launch_count() == (2 if behind else 1)
    head, count = want["state"]
    assert count == 30 - 7 + 10 and want["status"] & step.BAD_LENGTH
    free = {t.ring.tolist()[(head + i) % size] for i in range(count)}
    served = t.table.cpu().numpy()
    assert not free & {int(served[s, i]) for s in (0, 2, 4) for i in range(want["held"][s])}


def test_tables_rows_behind_the_last_sequence():
    t = Tables(kept=[5, 40], new=[3, 2], held=[1, 3], table=[[2, 0, 0], [1, 0, 3]], ring=[9, 9, 9, 9], state=[0, 0], n_rows=600)
    t.call()
    want = t.check()
    assert want["slots"][5:] == [-1] * 595


@pytest.mark.parametrize("rows", [3, 2000])
def test_tables_graph_replays_follow_the_lengths(rows):
    """A captured call in place, replayed over several steps, each compared."""
    n = 12
    t = Tables(**batch(31, n=n, rows=rows, spare=40 * n + rows * n))
    kept, state = t.kept.clone(), t.state.clone()

    def call():
        t.kvrp.kv_step_tables(t.kept, t.new, t.seqs, held_pages=t.held, free_pages=t.ring, free_state=t.state,
                              positions=t.positions, slots=t.slots, d_status=t.status)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    assert torch.equal(kept, t.kept) and torch.equal(state, t.state)
    rng = np.random.default_rng(5)
    for i in range(6):
        t.status.zero_()
        graph.replay()
        want = t.check(held=t.held, state=t.state)
        assert i or want["status"] == 0   # later steps of 2000 rows come to the tables' ends
        lens = np.array(want["seq_lens"])
        lens = np.maximum(lens - rng.integers(0, 20, n), 0) * (rng.random(n) > 0.15)
        t.host.update(kept=lens, table=want["table"], ring=want["ring"], state=want["state"], held=want["held"],
                      new=np.array(t.host["new"]) * (lens > 0))
        t.kept.copy_(i32(t.host["kept"]))
        t.new.copy_(i32(t.host["new"]))


# --- verification ----------------------------------------------------------------------
class Verify:
    def __init__(self, rows, vocab, bf16=False, draft=True, seed=0, pad=0, skew=(0, 0), lens=None, likely=0.5):
        import position_invariant_kv_gb300 as kvrp
        self.kvrp, self.rows, self.vocab, self.certain, self.bf16 = kvrp, rows, vocab, not draft, bf16
        rng = np.random.default_rng(seed)
        n, kind = sum(rows), torch.bfloat16 if bf16 else torch.float32
        self.n, self.stride = n, vocab + pad
        logits = 2 * rng.standard_normal((n, vocab))
        near = logits + likely * rng.standard_normal((n, vocab))
        soft = lambda x: np.exp(x - x.max(-1, keepdims=True)) / np.exp(x - x.max(-1, keepdims=True)).sum(-1, keepdims=True)  # noqa: E731
        self.p, self.q = (torch.tensor(soft(x), dtype=torch.float32).to(kind) for x in (logits, near))
        self.tokens = np.zeros(n, np.int64)
        for r in range(n - 1):
            w = self.q[r].double().numpy()
            self.tokens[r + 1] = w.argmax() if self.certain and rng.random() < 0.7 else rng.choice(vocab, p=w / w.sum())
        self.u, self.v = rng.random(n).astype(np.float32), rng.random(len(rows)).astype(np.float32)
        self.u = np.minimum(self.u, np.float32(1 - 2.0 ** -24))
        self.v = np.minimum(self.v, np.float32(1 - 2.0 ** -24))
        self.lens = [r + 3 for r in rows] if lens is None else lens
        self.skew = skew

    def place(self, x, skew):
        """x's rows at the stride, the first `skew` elements past an aligned address; NaN in between."""
        flat = torch.full((skew + self.n * self.stride + 8,), float("nan"), dtype=x.dtype, device="cuda")
        view = flat[skew:skew + self.n * self.stride].view(self.n, self.stride)
        view[:, :self.vocab] = x.cuda()
        return view

    def call(self, lens=None, in_place=False, stream=None):
        starts = np.concatenate([[0], np.cumsum(self.rows)])
        self.d_lens = i32(self.lens)
        self.seqs = self.kvrp.Seqs(seq_lens=self.d_lens, block_tables=torch.zeros((len(self.rows), 400), dtype=torch.int32, device="cuda"),
                                   num_pages=1, n_rows=self.n, row_start=i32(starts))
        self.out, self.accepted = i32([-9] * self.n), i32([-9] * len(self.rows))
        self.kept, self.in_place = self.d_lens if in_place else i32([-9] * len(self.rows)), in_place
        self.status = i32([0])
        self.args = dict(vocab=self.vocab, tokens=i32(self.tokens), u_accept=torch.tensor(self.u, device="cuda"),
                         u_sample=torch.tensor(self.v, device="cuda"), out_tokens=self.out, accepted=self.accepted,
                         kept_lens=self.kept, target_stride=self.stride, draft_stride=self.stride, d_status=self.status,
                         prob_type=self.kvrp.KVRP_BF16 if self.bf16 else self.kvrp.KVRP_F32)
        self.target = self.place(self.p, self.skew[0])
        self.draft = None if self.certain else self.place(self.q, self.skew[1])
        self.kvrp.kv_verify_drafts(self.target, self.seqs, draft=self.draft, stream=stream, **self.args)

    def want(self):
        out, accepted, kept, odd, at = [], [], [], False, 0
        p, q = self.p.float().numpy(), self.q.float().numpy()
        for r, v, length in zip(self.rows, self.v, self.lens):
            if r and length:
                a, token, o = step.verify_sequence(p[at:at + r], None if self.certain else q[at:at + r], self.tokens[at:at + r],
                                                   self.u[at:at + r], v)
                out += [int(x) for x in self.tokens[at + 1:at + 1 + a]] + [token] + [-1] * (r - 1 - a)
                accepted.append(a)
                kept.append(length - (r - 1 - a))
                odd |= o
            else:
                out += [-1] * r
                accepted.append(0)
                kept.append(length if length or self.in_place else -9)   # an idle place's stays
            at += r
        return out, accepted, kept, odd

    def check(self):
        torch.cuda.synchronize()
        out, accepted, kept, odd = self.want()
        assert self.accepted.tolist() == accepted
        assert self.out.tolist() == out
        assert self.kept.tolist() == kept
        assert int(self.status) == (step.BAD_TOKEN if odd else 0)
        return accepted


VERIFY = {
    "one": dict(rows=[5], vocab=32000), "one_certain": dict(rows=[5], vocab=32000, draft=False),
    "batch": dict(rows=[4, 1, 3, 5, 2, 0, 4], vocab=4099), "batch_bf16": dict(rows=[4, 1, 3, 5, 2, 0, 4], vocab=4099, bf16=True),
    "certain_bf16": dict(rows=[3, 2, 6], vocab=1777, bf16=True, draft=False),
    "odd_large": dict(rows=[3, 2], vocab=130003), "odd_large_bf16": dict(rows=[3, 2], vocab=130003, bf16=True),
    "one_token": dict(rows=[2, 1], vocab=1), "three": dict(rows=[3, 3, 1, 2], vocab=3), "thirty_one": dict(rows=[4, 4], vocab=31, pad=5),
    "strides": dict(rows=[3, 4, 2], vocab=2049, pad=7, skew=(1, 3)), "strides_bf16": dict(rows=[3, 4, 2], vocab=2049, pad=7, skew=(5, 2), bf16=True),
    "aligned": dict(rows=[3, 4, 2], vocab=8192), "long_drafts": dict(rows=[70, 34, 33], vocab=61, likely=0.05),
    "close": dict(rows=[9] * 20, vocab=509, likely=0.1), "idle": dict(rows=[3, 2, 1, 2], vocab=300, lens=[9, 0, 5, 0]),
    "many": dict(rows=[2] * 700, vocab=40),
}


@pytest.mark.parametrize("seed", [0, 1])
@pytest.mark.parametrize("name", list(VERIFY))
def test_verify(name, seed):
    x = Verify(seed=50 + seed, **VERIFY[name])
    x.call(in_place=seed == 1)
    x.check()


@pytest.mark.parametrize("bf16", [False, True])
def test_verify_numbers_at_their_ends(bf16):
    """u of 0, the largest below 1, and out of range; draws on the border of two tokens."""
    x = Verify([1] * 10, 1030, bf16=bf16, seed=4)
    x.p[:] = 0
    x.p[:, [5, 500, 1029]] = torch.tensor([0.25, 0.5, 0.25], dtype=x.p.dtype)
    x.v = np.array([0, 0.25 - 2 ** -26, 0.25, 0.75 - 2 ** -24, 0.75, 1 - 2 ** -24, 1, -1, np.nan, 2], np.float32)
    x.call()
    x.check()
    assert x.out.tolist() == [5, 5, 500, 500, 1029, 1029, 1029, 5, 5, 1029]


def test_verify_draft_turned_down_at_the_border():
    x = Verify([2] * 3, 64, seed=4)
    x.p[:], x.q[:] = 1 / 64, 0
    x.p[:, 7], x.q[:, 7] = 0.25, 0.5
    x.tokens[1::2] = 7
    x.u[::2] = [0.5, 0.5 - 2.0 ** -25, 0.5 + 2.0 ** -24]
    x.call()
    assert x.check() == [0, 1, 0]


@pytest.mark.parametrize("draft", [True, False])
def test_verify_odd_values(draft):
    """NaN, infinities, negative values, rows without weight or without a positive part, tokens out of range."""
    x = Verify([3] * 12, 777, draft=draft, seed=9)
    p, q = x.p, x.q
    p[0, 3], p[1, 700], p[2, 5] = float("nan"), float("inf"), -1.0
    q[3, 1], q[4, :] = float("nan"), float("inf")
    p[6:9] = 0
    p[9:12] = float("nan")
    q[12:15] = 1
    p[15:18], q[15:18] = p[0].clone().nan_to_num(0.01), p[0].clone().nan_to_num(0.01)
    p[18, :] = 0
    x.tokens[19], x.tokens[22], x.tokens[25] = -1, 777, 2 ** 31 - 1
    p[27:30] = 2.0 ** -60
    x.call()
    x.check()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("draft", [True, False])
def test_verify_reads_the_type_off_the_tensors(bf16, draft):
    x = Verify([3, 2, 4], 777, bf16=bf16, draft=draft, seed=12)
    x.call()
    x.check()
    del x.args["prob_type"]
    x.out.fill_(-9)
    x.kvrp.kv_verify_drafts(x.target, x.seqs, draft=x.draft, **x.args)
    x.check()


def test_verify_bad_lengths_keep_their_outputs():
    x = Verify([3, 4, 2, 2], 500, seed=3)
    x.lens = [9, 3, -1, 8]            # fewer tokens than rows; a negative length
    x.call()
    torch.cuda.synchronize()
    assert int(x.status) == step.BAD_LENGTH
    assert x.out[3:9].tolist() == [-9] * 6 and x.accepted[1:3].tolist() == [-9, -9] and x.kept[1:3].tolist() == [-9, -9]
    x.lens = [9, 9, 9, 8]
    out, accepted, kept, _ = x.want()
    assert x.out[:3].tolist() == out[:3] and x.out[9:].tolist() == out[9:] and x.accepted[[0, 3]].tolist() == [accepted[0], accepted[3]]


def test_verify_graph_and_streams():
    """Two captured calls replayed on two streams at once, over new numbers each time."""
    xs = [Verify([4] * 9, 3001, seed=i, draft=i == 0) for i in range(2)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, st in zip(xs, streams):
        x.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            x.kvrp.kv_verify_drafts(x.target, x.seqs, draft=x.draft, **x.args)
        graphs.append(g)
    rng = np.random.default_rng(0)
    for _ in range(5):
        for x in xs:
            x.u, x.v = rng.random(x.n).astype(np.float32), rng.random(len(x.rows)).astype(np.float32)
            x.args["u_accept"].copy_(torch.tensor(x.u))
            x.args["u_sample"].copy_(torch.tensor(x.v))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        for x in xs:
            x.check()


def test_verify_rows_past_32_bits():
    """Rows 2^30 elements and one apart: element, and byte, offsets past 2^31."""
    x = Verify([4, 1], 1003, bf16=True, seed=6, pad=2 ** 30 - 1002)
    x.call()
    x.check()


def test_a_sequence_without_pages_goes_on_when_there_are_some():
    """Tables and verification in turn: one that could not be served keeps its tokens, then gets its page."""
    t = Tables(kept=[15, 31], new=[2, 2], held=[1, 2], table=[[0, -1, -1], [1, 2, -1]], ring=[3, -1, -1, -1, -1], state=[0, 1])
    t.call(held_out=t.held, free_state_out=t.state)
    assert t.check(held=t.held, state=t.state)["status"] == step.NO_PAGES
    out, accepted, kept = i32([-9] * 4), i32([-9] * 2), t.kept
    target = torch.full((4, 8), 0.125, device="cuda")
    t.kvrp.kv_verify_drafts(target, t.seqs, vocab=8, tokens=i32([1, 2, 3, 4]), u_accept=torch.zeros(4, device="cuda"),
                            u_sample=torch.zeros(2, device="cuda"), out_tokens=out, accepted=accepted, kept_lens=kept,
                            d_status=t.status)
    assert kept.tolist() == [17, 31] and accepted.tolist() == [1, 0] and out.tolist() == [2, 0, -1, -1]
    t.ring[1], t.state[1] = 4, 1                  # a page has become free
    t.host.update(kept=[17, 31], table=t.table.cpu().numpy(), ring=t.ring.tolist(), state=t.state.tolist(), held=t.held.tolist())
    t.status.zero_()
    t.call(held_out=t.held, free_state_out=t.state)
    want = t.check(held=t.held, state=t.state)
    assert want["status"] == 0 and want["seq_lens"] == [19, 33] and t.table[1].tolist() == [1, 2, 4]
