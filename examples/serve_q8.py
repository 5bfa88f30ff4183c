"""One layer of a serving step on top of reused chunks, end to end.

    python examples/serve_q8.py

Two chunks that were cached on their own are relocated behind each other into the paged
bf16 cache (kv_relocate_batch), moved into the 8-bit cache (kv_pack_q8), and two sequences
go on over them: a question's rows are normed, rotated and appended (kv_append_q8) and
attend over chunks and question (kv_attend_q8); then tokens are decoded one at a time from
a captured CUDA graph that follows the lengths on the device.  Every attention output is
compared with the fp32 evaluation over the same 8-bit cache.

The queries, keys and values of new rows are random: they stand in for a model's
projections.  Needs a GB300.
"""
from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch

import position_invariant_kv_gb300 as kvrp

HQ, HKV, D, THETA = 28, 4, 128, 1e6
CHUNK, QUESTION, DECODE, SEQS = 500, 37, 20, 2
ROW = HKV * D
SAME = dict(n_q_heads=HQ, n_kv_heads=HKV, head_dim=D)


def i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def plain_attention(q, length, rows, table, k_pool, k_scale, v_pool, v_scale):
    """softmax(q K^T / sqrt(d)) V in fp32 for the last `rows` of `length` tokens."""
    k, v = ((p[table.long()].float() * s[table.long()][:, None, :, None]).reshape(-1, HKV, D)[:length]
            for p, s in ((k_pool, k_scale), (v_pool, v_scale)))
    k, v = (x.repeat_interleave(HQ // HKV, 1) for x in (k, v))
    s = torch.einsum("rhd,thd->hrt", q.float(), k) * D ** -0.5
    later = torch.arange(length, device="cuda")[None] > torch.arange(length - rows, length, device="cuda")[:, None]
    return torch.einsum("hrt,thd->rhd", torch.softmax(s.masked_fill(later, float("-inf")), -1), v)


def main() -> None:
    torch.manual_seed(7)
    bf = dict(dtype=torch.bfloat16, device="cuda")
    pages_each = -(-(2 * CHUNK + QUESTION + DECODE) // 16)
    pages = SEQS * pages_each + 3
    tables = torch.randperm(pages, device="cuda")[: SEQS * pages_each].to(torch.int32).view(SEQS, pages_each).contiguous()
    status = i32([0])

    # 1. the chunks of both sequences, relocated into the bf16 pages of the layer
    canon = torch.randn(2, 2, CHUNK, ROW, **bf)                        # [chunk][K, V]
    k16, v16 = (torch.zeros(pages, 16, ROW, **bf) for _ in range(2))
    chunks = []
    for s in range(SEQS):
        for c in range(2):
            at = dict(num_pages=pages, block_table=tables[s], dst_start=c * CHUNK)
            chunks.append(kvrp.Chunk(k_src=canon[c, 0], v_src=canon[c, 1], n_tokens=CHUNK, delta=c * CHUNK - 40 * s,
                                     k_dst=kvrp.Dst(base=k16, **at), v_dst=kvrp.Dst(base=v16, **at)))
    ws = torch.empty(kvrp.kv_relocate_batch_workspace_size(len(chunks)), dtype=torch.uint8, device="cuda")
    kvrp.kv_relocate_batch(chunks, n_layers=1, n_kv_heads=HKV, head_dim=D, rope_theta=THETA, workspace=ws, d_status=status)

    # 2. into the 8-bit cache, page by page
    k_pool, v_pool = (torch.zeros(pages, 16, HKV, D, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    k_scale, v_scale = (torch.ones(pages, HKV, device="cuda") for _ in range(2))
    cache = dict(k_pool=k_pool, v_pool=v_pool, k_scale=k_scale, v_scale=v_scale)
    for s in range(SEQS):
        kvrp.kv_pack_q8(k16, v16, n_layers=1, n_tokens=2 * CHUNK, n_kv_heads=HKV, head_dim=D, src_table=tables[s],
                        src_pages=pages, block_table=tables[s], num_pages=pages, d_status=status, **cache)

    # 3. the questions: a ragged batch of new rows behind the chunks
    rows = [QUESTION, QUESTION - 9]
    lens = [2 * CHUNK + r for r in rows]
    q_norm, k_norm = torch.ones(D, **bf), torch.ones(D, **bf)

    def step(qkv, seqs, q, out, workspace):
        kvrp.kv_append_q8(qkv[:, :HQ], qkv[:, HQ:HQ + HKV], qkv[:, HQ + HKV:], seqs, **SAME, rope_theta=THETA, q_out=q,
                          q_norm=q_norm, k_norm=k_norm, q_stride=qkv.stride(0), k_stride=qkv.stride(0),
                          v_stride=qkv.stride(0), d_status=status, **cache)
        kvrp.kv_attend_q8(q, seqs, **SAME, softmax_scale=D ** -0.5, out=out, workspace=workspace, d_status=status, **cache)

    def check(what, q, out, lens, rows):
        torch.cuda.synchronize()
        at, worst = 0, 0.0
        for s in range(SEQS):
            ref = plain_attention(q[at:at + rows[s]], lens[s], rows[s], tables[s], k_pool, k_scale, v_pool, v_scale)
            worst = max(worst, ((out[at:at + rows[s]].float() - ref).norm() / ref.norm()).item())
            at += rows[s]
        assert int(status) == 0 and worst < 5e-3, (what, int(status), worst)   # bf16 rounding is 1.7e-3 of it
        print(f"{what}: relative difference to the plain evaluation {worst:.1e}")

    n = sum(rows)
    seqs = kvrp.Seqs(seq_lens=i32(lens), block_tables=tables, num_pages=pages, n_rows=n,
                     row_start=i32([0, rows[0], n]), max_rows=max(rows))
    workspace = torch.empty(kvrp.kv_attend_q8_workspace_size(HQ, HKV, D, max(rows)), dtype=torch.uint8, device="cuda")
    q, out = torch.empty(n, HQ, D, **bf), torch.empty(n, HQ, D, **bf)
    step(torch.randn(n, HQ + 2 * HKV, D, **bf), seqs, q, out, workspace)
    check("questions behind two reused chunks", q, out, lens, rows)

    # 4. decode: one graph, replayed while the lengths advance on the device
    d_lens = i32([x + 1 for x in lens])
    seqs = kvrp.Seqs(seq_lens=d_lens, block_tables=tables, num_pages=pages)
    workspace = torch.empty(kvrp.kv_attend_q8_workspace_size(HQ, HKV, D, 1), dtype=torch.uint8, device="cuda")
    qkv = torch.randn(SEQS, HQ + 2 * HKV, D, **bf)
    q, out = torch.empty(SEQS, HQ, D, **bf), torch.empty(SEQS, HQ, D, **bf)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step(qkv, seqs, q, out, workspace)
    for i in range(DECODE):
        qkv.copy_(torch.randn(SEQS, HQ + 2 * HKV, D, **bf))
        if i:
            d_lens.add_(1)
        graph.replay()
        lens = [x + 1 for x in lens]
    check(f"{DECODE} decoded tokens from a graph", q, out, lens, [1] * SEQS)


if __name__ == "__main__":
    main()
