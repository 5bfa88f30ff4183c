"""kv_verify_drafts where a cluster of CTAs takes a sequence: the paths that the small vocabularies of
test_gpu_step.py run in one CTA.  A sequence has one CTA for each 4096 tokens, at most eight.

All outputs are whole numbers, so every comparison is for equality with the oracle."""
import numpy as np
import pytest
import torch

from oracle import step
from test_gpu_step import Verify, gpu  # noqa: F401

pytestmark = pytest.mark.gpu

VOCAB = 33001                       # eight CTAs
ROWS = dict(pad=3, skew=(1, 2))     # rows that begin off 16 bytes, target's and draft's differently


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("draft", [True, False])
def test_no_positive_part(draft, bf16):
    """Every draft is turned down and leaves nothing to draw from: the second try goes over all CTAs, and the tokens
    that are drawn lie in all parts of the row."""
    n = 16
    x = Verify([2] * n, VOCAB, bf16=bf16, draft=draft, seed=21, **ROWS)
    x.u[:] = 0.9
    x.v = (np.arange(n) / n + 2.0 ** -8).astype(np.float32)
    if draft:
        x.q = (2 * x.p.float()).clamp(max=1).to(x.p.dtype)   # exactly twice the target: 0.9 q is not below p
    else:
        x.p[:] = 0
        x.tokens[1::2] = np.arange(n) * (VOCAB - 1) // (n - 1)
        x.p[torch.arange(0, 2 * n, 2), torch.as_tensor(x.tokens[1::2])] = 0.5   # the drafted token is all there is
    x.call()
    assert x.check() == [0] * n
    drawn = x.out[::2].cpu().numpy()
    assert len(set(drawn * 8 // VOCAB)) >= 7
    if not draft:
        assert drawn.tolist() == x.tokens[1::2].tolist()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("draft", [True, False])
def test_odd_values(draft, bf16):
    """NaN, infinities, negative values, rows without weight, tokens out of range."""
    x = Verify([3] * 12, VOCAB, bf16=bf16, draft=draft, seed=9, **ROWS)
    p, q = x.p, x.q
    p[0, 30003], p[1, 20700], p[2, 5] = float("nan"), float("inf"), -1.0
    q[3, 12001], q[4, :] = float("nan"), float("inf")
    p[6:9] = 0
    p[9:12] = float("nan")
    q[12:15] = 1
    p[18, :] = 0
    x.tokens[19], x.tokens[22], x.tokens[25] = -1, VOCAB, 2 ** 31 - 1
    p[27:30] = 2.0 ** -60
    p[33:36] = 0
    p[33:36, VOCAB - 1] = 1      # the last token of the last CTA is all there is
    x.call()
    x.check()


@pytest.mark.parametrize("bf16", [False, True])
@pytest.mark.parametrize("in_place", [False, True])
def test_idle_places_and_sequences_without_rows(in_place, bf16):
    x = Verify([3, 2, 0, 1, 0, 2, 4], VOCAB, bf16=bf16, seed=5, lens=[9, 0, 7, 5, 0, 0, 8], **ROWS)
    x.call(in_place=in_place)
    x.check()


def test_bad_lengths_keep_their_outputs():
    x = Verify([3, 4, 2, 2], VOCAB, seed=3, **ROWS)
    x.lens = [9, 3, -1, 8]            # fewer tokens than rows; a negative length
    x.call()
    torch.cuda.synchronize()
    assert int(x.status) == step.BAD_LENGTH
    assert x.out[3:9].tolist() == [-9] * 6 and x.accepted[1:3].tolist() == [-9, -9] and x.kept[1:3].tolist() == [-9, -9]
    x.lens = [9, 9, 9, 8]
    out, accepted, kept, _ = x.want()
    assert x.out[:3].tolist() == out[:3] and x.out[9:].tolist() == out[9:] and x.accepted[[0, 3]].tolist() == [accepted[0], accepted[3]]
    assert x.kept[[0, 3]].tolist() == [kept[0], kept[3]]


def test_two_graphs_at_once():
    """Captured calls replayed on two streams, over new numbers each time."""
    xs = [Verify([4] * 9, VOCAB, seed=i, draft=i == 0, **ROWS) for i in range(2)]
    graphs, streams = [], [torch.cuda.Stream(), torch.cuda.Stream()]
    for x, st in zip(xs, streams):
        x.call()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=st):
            x.kvrp.kv_verify_drafts(x.target, x.seqs, draft=x.draft, **x.args)
        graphs.append(g)
    rng = np.random.default_rng(0)
    for _ in range(4):
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


@pytest.mark.parametrize("n, vocab", [(40, 9001), (3, 4096 * 5 + 3), (160, 8192), (1, 4095)])
def test_other_numbers_of_ctas(n, vocab):
    """Two, five, two (many sequences) and one CTA a sequence."""
    x = Verify([1 + i % 3 for i in range(n)], vocab, seed=n, likely=0.9, **ROWS)
    x.call()
    x.check()
