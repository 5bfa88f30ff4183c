"""Small seeded batches for the tests of the serving calls: bf16 rows, block
tables over a shuffled pool, and the caches as NumPy and torch see them."""
from __future__ import annotations

import numpy as np
import torch

from oracle import bf16_bits_to_f64, round_to_bf16_bits


def dev(bits):
    return torch.from_numpy(np.ascontiguousarray(bits).view(np.int16)).cuda().view(torch.bfloat16)


def f64(t):
    """A bf16, float8 or fp32 tensor's values in fp64."""
    return t.detach().to(torch.float32).cpu().numpy().astype(np.float64)


def bf16(rng, shape, size=1.0):
    return round_to_bf16_bits(size * rng.standard_normal(shape))


def i32(x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def layout(rng, ctx, rows, spare=3):
    """Lengths, row starts and shuffled block tables of sequences with ctx[s] cached
    tokens and rows[s] new ones; unused table entries are -1 (never read)."""
    lens = [a + b for a, b in zip(ctx, rows)]
    need = [-(-n // 16) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    table = np.full((len(ctx), max(need + [1]) + 1), -1, np.int32)
    at = 0
    for s, n in enumerate(need):
        table[s, :n] = order[at:at + n]
        at += n
    starts = np.concatenate([[0], np.cumsum(rows)]).astype(np.int32)
    return lens, starts, table, pages


__all__ = ["dev", "f64", "bf16", "i32", "layout", "bf16_bits_to_f64"]
