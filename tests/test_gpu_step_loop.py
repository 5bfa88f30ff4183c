"""The calls of a step together, as a decode loop uses them: tables, append, attention over the shared
and the own tokens, verification, captured in one graph and replayed while sequences grow, end and begin.

Every replay is compared with the oracles: tables, lengths, positions, slots, rings and tokens for
equality (oracle/step.py), attention element by element over the cache as it then is (oracle/serve.py),
with the bars of test_gpu_attend_q8.py: scores here are below 16 in magnitude sums as there."""
import numpy as np
import pytest
import torch

from oracle import step
from oracle.serve import attend_rows, e4m3_round, q8_scale
from serve_util import f64, i32

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from position_invariant_kv_gb300.build import build
    build()


def e4m3(x):
    return torch.from_numpy(x.astype(np.float32)).to(torch.float8_e4m3fn).view(torch.uint8)


@pytest.mark.parametrize("each", [0, -1])
@pytest.mark.parametrize("hq,hkv,d,rows", [(8, 2, 128, 4), (14, 2, 64, 4), (4, 4, 128, 1), (32, 2, 64, 5)])
def test_a_decode_loop(hq, hkv, d, rows, each):
    """4 rows x group 4: the kernel for few rows; x group 7: in runs; 5 rows x group 16: the kernel for many.
    each 0: the shared pages are read once for the batch; -1: few as they are here, by each sequence."""
    import position_invariant_kv_gb300 as kvrp
    kvrp.kvrp_test_set_each_limit(each)
    try:
        decode_loop(kvrp, hq, hkv, d, rows)
    finally:
        kvrp.kvrp_test_set_each_limit(-1)


def decode_loop(kvrp, hq, hkv, d, rows):
    rng = np.random.default_rng(rows * d + hq)
    n, vocab, shared, steps = 6, 501, 5, 7
    pages, stride = shared + 40, shared + 9
    order = rng.permutation(pages)
    table = np.full((n, stride), -1)
    ring, state = np.full(pages, -1), np.array([11, pages - shared])
    ring[(state[0] + np.arange(state[1])) % pages] = order[shared:]
    prefix_table, prefix_len = order[:shared], 16 * shared + 7
    kept, new, held = np.full(n, 16 * shared), np.full(n, rows), np.zeros(n, int)
    kept[2] = new[2] = 0                                         # a place that is free at first

    # the cache: the shared pages hold tokens, the others anything
    pools, scales = [], []
    for _ in range(2):
        x = rng.standard_normal((pages, 16, hkv, d))
        s = np.array([[q8_scale(x[p, :, h]) for h in range(hkv)] for p in range(pages)])
        raw = e4m3(e4m3_round(x / s[:, None, :, None]))
        raw[torch.from_numpy(order[shared:])] = 0x7F
        pools.append(raw.cuda())
        scales.append(torch.from_numpy(s.astype(np.float32)).cuda())
    cache = dict(k_pool=pools[0], v_pool=pools[1], k_scale=scales[0], v_scale=scales[1])
    same = dict(n_q_heads=hq, n_kv_heads=hkv, head_dim=d)
    total = n * rows
    dev = dict(device="cuda")
    d_kept, d_new, d_held, d_ring, d_state, d_table = (i32(x) for x in (kept, new, held, ring, state, table))
    d_lens, d_starts, status = i32([0] * n), i32([0] * (n + 1)), i32([0])
    positions, slots = torch.zeros(total, dtype=torch.int32, **dev), torch.zeros(total, dtype=torch.int64, **dev)
    seqs = kvrp.Seqs(seq_lens=d_lens, block_tables=d_table, num_pages=pages, n_rows=total, row_start=d_starts, max_rows=rows)
    prefix = kvrp.Prefix(i32(prefix_table), i32([prefix_len]))
    qkv = torch.zeros((total, hq + 2 * hkv, d), dtype=torch.bfloat16, **dev)
    q, out = (torch.zeros((total, hq, d), dtype=torch.bfloat16, **dev) for _ in range(2))
    target, draft = (torch.zeros((total, vocab), **dev) for _ in range(2))
    tokens, out_tokens = (torch.zeros(total, dtype=torch.int32, **dev) for _ in range(2))
    u_accept, u_sample, accepted = torch.zeros(total, **dev), torch.zeros(n, **dev), i32([0] * n)
    ws = torch.full((kvrp.kv_attend_shared_q8_workspace_size(hq, hkv, d, rows, total),), 0xFF, dtype=torch.uint8, **dev)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kvrp.kv_step_tables(d_kept, d_new, seqs, held_pages=d_held, free_pages=d_ring, free_state=d_state, prefix=prefix,
                            positions=positions, slots=slots, d_status=status)
        kvrp.kv_append_q8(qkv[:, :hq], qkv[:, hq:hq + hkv], qkv[:, hq + hkv:], seqs, **same, rope_theta=1e4, q_out=q,
                          q_stride=qkv.stride(0), k_stride=qkv.stride(0), v_stride=qkv.stride(0), positions=positions,
                          d_status=status, **cache)
        kvrp.kv_attend_shared_q8(q, seqs, prefix, **same, softmax_scale=d ** -0.5, out=out, workspace=ws, d_status=status, **cache)
        kvrp.kv_verify_drafts(target, seqs, vocab=vocab, draft=draft, tokens=tokens, u_accept=u_accept, u_sample=u_sample,
                              out_tokens=out_tokens, accepted=accepted, kept_lens=d_kept, d_status=status)
    for i in range(steps):
        # inputs of the step
        qkv.copy_(torch.from_numpy(0.7 * rng.standard_normal(tuple(qkv.shape))).to(torch.bfloat16))
        logits = 2 * rng.standard_normal((total, vocab))
        soft = lambda x: (np.exp(x) / np.exp(x).sum(-1, keepdims=True)).astype(np.float32)  # noqa: E731
        p, pq = soft(logits), soft(logits + 0.4 * rng.standard_normal(logits.shape))
        tok = np.concatenate([[0], [rng.choice(vocab, p=w.astype(np.float64) / w.astype(np.float64).sum()) for w in pq[:-1]]])
        ua, us = (np.minimum(rng.random(m).astype(np.float32), np.float32(1 - 2.0 ** -24)) for m in (total, n))
        for t, x in ((target, p), (draft, pq), (tokens, tok.astype(np.int32)), (u_accept, ua), (u_sample, us)):
            t.copy_(torch.from_numpy(x))
        graph.replay()
        torch.cuda.synchronize()
        # tables
        want = step.step_tables(kept, new, held, table, ring, state, total, prefix_table, prefix_len)
        assert want["status"] == 0 and int(status) == 0
        for name, t in (("table", d_table), ("ring", d_ring), ("held", d_held), ("state", d_state), ("row_start", d_starts),
                        ("seq_lens", d_lens), ("positions", positions), ("slots", slots)):
            assert np.array_equal(t.cpu().numpy(), np.array(want[name]).reshape(t.shape)), (i, name)
        table, ring, held, state = want["table"], want["ring"], want["held"], want["state"]
        lens, starts = want["seq_lens"], want["row_start"]
        # attention and tokens, over the cache as it is now
        values = [x.view(torch.float8_e4m3fn).float().cpu().numpy() * s.cpu().numpy()[:, None, :, None] for x, s in zip(pools, scales)]
        got, qs = f64(out), f64(q)
        got_tokens, got_accepted, got_kept = out_tokens.tolist(), accepted.tolist(), d_kept.tolist()
        kept = np.zeros(n, int)
        for s in range(n):
            a, b = starts[s], starts[s + 1]
            if a == b:
                assert lens[s] == 0 and got_accepted[s] == 0 and got_kept[s] == 0
                continue
            t = np.arange(lens[s])
            k, v = (x[table[s][t // 16], t % 16].astype(np.float64) for x in values)
            ref, _, mag = attend_rows(qs[a:b], k, v, hkv, d ** -0.5)
            assert (d ** -0.5 * np.abs(qs[a:b]).reshape(b - a, hkv, -1, d) @ np.abs(k).transpose(1, 2, 0)[None]).max() < 16
            assert np.all(np.abs(got[a:b] - ref) <= 2.0 ** -8 * np.abs(ref) + 2.0 ** -10 * mag), (i, s)
            stay, token, odd = step.verify_sequence(p[a:b], pq[a:b], tok[a:b], ua[a:b], us[s])
            assert got_tokens[a:b] == [int(x) for x in tok[a + 1:a + 1 + stay]] + [token] + [-1] * (b - a - 1 - stay)
            kept[s] = lens[s] - (b - a - 1 - stay)
            assert (got_accepted[s], got_kept[s], odd) == (stay, kept[s], False)
        # one sequence ends, another begins in a free place
        if i == 2:
            kept[4] = new[4] = 0
            kept[2], new[2] = 16 * shared, rows
        if i == 4:
            kept[4], new[4] = 16 * shared, rows
        d_kept.copy_(i32(kept))
        d_new.copy_(i32(new))
