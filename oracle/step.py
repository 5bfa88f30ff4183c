"""The step around attention: batch tables and draft verification (oracle; test
infrastructure only).

Plain definitions, a sequence at a time in Python's whole numbers:

* tables: a sequence with `kept` tokens in the cache and `new` rows needs
  ceil((kept + new) / 16) pages; the first `shared` are the prefix's, the others its
  own, taken from a ring of free pages and given back behind it;
* drafts: a draft stays while u q < p; the token after the last one that does is
  drawn from the positive part of p - q, in whole numbers of 2^-40.
"""
from __future__ import annotations

from fractions import Fraction

import numpy as np

PAGE = 16
BAD_PAGE, BAD_LENGTH, NO_PAGES, BAD_TOKEN = 0x1, 0x4, 0x8, 0x10


def step_tables(kept, new, held, table, ring, state, n_rows, prefix_table=(), prefix_len=0):
    """What kv_step_tables writes, as a dict; table and ring are copied."""
    table, ring, size = np.array(table, np.int64), [int(x) for x in ring], len(ring)
    stride, (head, count) = table.shape[1], (int(x) for x in state)
    shared, status = int(prefix_len) // PAGE, 0
    usable = 0 <= head < size and 0 <= count <= size and prefix_len >= 0 and shared <= len(prefix_table)
    if not usable:
        status |= BAD_LENGTH
    asked = taken = given = at = 0
    starts, lens, left = [0], [], [int(x) for x in held]
    positions, slots = [0] * n_rows, [-1] * n_rows
    taking = dict(enumerate(ring))   # the ring as it was: what is given back is not taken in the same call
    for s, (k, m, h) in enumerate(zip(kept, new, held)):
        k, m, h = int(k), int(m), int(h)
        length, start = k + m, at
        at += max(m, 0)
        starts.append(min(at, n_rows))
        fine = usable and k >= 0 and m >= 0 and 0 <= h <= stride and (h == 0 or h >= shared) and at <= n_rows
        fine = fine and length <= stride * PAGE and length <= 0x7fffff00
        if fine and length:
            fine = shared * PAGE <= k <= max(h, shared) * PAGE
        need = -(-length // PAGE) if fine else 0
        takes = max(0, need - max(h, shared)) if need else 0
        asked += takes
        served = fine and (takes == 0 or asked <= count)
        if not served:
            status |= NO_PAGES if fine else BAD_LENGTH
            lens.append(0)
            continue
        for e in range(h, need):
            if e < shared:
                page = int(prefix_table[e])
            else:
                page = taking[(head + taken) % size]
                taken += 1
            table[s, e] = page
            status |= 0 if 0 <= page < size else BAD_PAGE
        for e in range(max(need, shared), h):
            status |= 0 if 0 <= table[s, e] < size else BAD_PAGE
            if count + given < size:
                ring[(head + count + given) % size] = int(table[s, e])
                given += 1
            else:
                status |= BAD_LENGTH   # lost: no place, and not counted
        for i in range(m):
            page = int(table[s, (k + i) // PAGE])
            positions[start + i] = k + i
            if 0 <= page < size:
                slots[start + i] = page * PAGE + (k + i) % PAGE
            else:
                status |= BAD_PAGE
        left[s] = need
        lens.append(length)
    state = [(head + taken) % size, count - taken + given] if usable else [head, count]
    return {"table": table, "ring": ring, "state": state, "held": left, "row_start": starts, "seq_lens": lens,
            "positions": positions, "slots": slots, "status": status}


def whole(x):
    """Probabilities (fp32 values) as whole numbers of 2^-40: Python ints."""
    x = np.nan_to_num(np.asarray(x, np.float64), nan=0.0, posinf=1.0, neginf=0.0)
    return [int(v) for v in np.floor(np.clip(x, 0.0, 1.0) * 2.0 ** 40)]


def verify_sequence(target, draft, tokens, u_accept, u_sample):
    """One sequence: target [rows][vocab] (draft the same, or None), tokens and u_accept [rows].
    Returns (drafts that stay, drawn token or -1, whether a token was out of range or nothing weighed)."""
    rows, vocab = np.shape(target)
    for a in range(rows):
        if a == rows - 1:
            w, odd = whole(target[a]), False
            break
        t = int(tokens[a + 1])
        if not 0 <= t < vocab:
            stays = False
        else:
            p, q = float(target[a][t]), float(draft[a][t]) if draft is not None else 1.0
            if not all(np.isfinite((p, q))):
                stays = bool(np.float64(u_accept[a]) * q < p)
            else:
                stays = Fraction(float(u_accept[a])) * Fraction(q) < Fraction(p)
        if not stays:
            p = whole(target[a])
            if draft is not None:
                w = [max(0, x - y) for x, y in zip(p, whole(draft[a]))]
            else:
                w = [0 if i == t else x for i, x in enumerate(p)]
            w, odd = (w if sum(w) else p), not 0 <= t < vocab
            break
    total = sum(w)
    if not total:
        return a, -1, True
    u = float(u_sample)
    r = 0 if not u > 0 else min(int(u * 2.0 ** 32), 2 ** 32 - 1) if u < 1 else 2 ** 32 - 1
    threshold, upto = r * total >> 32, 0
    for i, x in enumerate(w):
        upto += x
        if upto > threshold:
            return a, i, odd
    raise AssertionError("the sum is above the threshold")
