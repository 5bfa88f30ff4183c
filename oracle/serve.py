"""Serving rows behind reused chunks: append, 8-bit cache and attention over it
(oracle; test infrastructure only).

After the chunks of a window were relocated (Kamera, gist.science/pt/paper/2606.23581,
section 3), new rows are normed, rotated, appended and attend over the cache.
Plain definitions in fp64:

* new rows: y = w x / sqrt(mean(x^2) + eps) per head, then rotate-half RoPE at
  the row's position (or M-RoPE, one position per section); values as they are;
* the 8-bit block: the 16 tokens x head_dim values of one (page, head) as e4m3
  values times 2^max(-126, ceil(log2(amax / 448)));
* appending into an open block: the larger of its scale and the new rows' one,
  the earlier values rounded again under it;
* attention: softmax(scale q K^T) V over the tokens up to the row's own position.
"""
from __future__ import annotations

import numpy as np

from .kamera import inv_freq

PAGE = 16
QMAX = 448.0
EMIN = -126


def _e4m3_values():
    """The 127 non-negative finite e4m3 values in order (4 exponent bits, bias 7, 3 mantissa bits, no inf)."""
    vals = []
    for code in range(127):
        e, m = code >> 3, code & 7
        vals.append(m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7))
    return np.array(vals)


E4M3 = _e4m3_values()


def e4m3_round(x):
    """x (fp64, |x| <= 448 or not finite) to the nearest e4m3 value, ties to the even code; not finite -> NaN."""
    x = np.asarray(x, dtype=np.float64)
    ok = np.isfinite(x)
    a = np.where(ok, np.abs(x), 0.0)
    hi = np.clip(np.searchsorted(E4M3, a), 0, 126)
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - E4M3[lo], E4M3[hi] - a
    code = np.where(dl < dh, lo, np.where(dh < dl, hi, np.where(lo % 2 == 0, lo, hi)))
    return np.where(ok, np.copysign(E4M3[code], x), np.nan)


def q8_scale(block) -> float:
    """The scale of a block's finite values: the least power of two s >= 2^-126 with amax <= 448 s."""
    b = np.abs(np.asarray(block, dtype=np.float64))
    amax = b[np.isfinite(b)].max(initial=0.0)
    if amax == 0.0:
        return 2.0 ** EMIN
    m, e = np.frexp(amax / QMAX)          # amax / 448 = m 2^e, m in [0.5, 1)
    e = int(e) - (1 if m == 0.5 else 0)
    if amax > QMAX * 2.0 ** e:            # amax / 448 rounded down onto the power of two
        e += 1
    elif e > EMIN and amax <= QMAX * 2.0 ** (e - 1):
        e -= 1
    return 2.0 ** max(EMIN, e)


def norm_rows(x, w, eps: float):
    """RMS norm over the last axis with weights w (x unchanged when w is None)."""
    if w is None:
        return np.asarray(x, dtype=np.float64)
    x = np.asarray(x, dtype=np.float64)
    return x / np.sqrt((x * x).mean(-1, keepdims=True) + eps) * np.asarray(w, dtype=np.float64)


def rotate_rows(x, positions, theta: float, sections=None):
    """x [rows][heads][d] turned by each row's position: positions [rows], or
    [3][rows] with M-RoPE sections (pairs per section)."""
    d = x.shape[-1]
    inv = inv_freq(d, theta)
    if sections is None:
        phi = np.outer(np.asarray(positions, dtype=np.float64), inv)
    else:
        sec = np.repeat(np.arange(3), sections)
        phi = np.asarray(positions, dtype=np.float64)[sec].T * inv
    c, s = np.cos(phi)[:, None], np.sin(phi)[:, None]
    a, b = x[..., : d // 2], x[..., d // 2:]
    return np.concatenate([a * c - b * s, b * c + a * s], axis=-1)


def rotate_magnitude(x, positions, theta: float, sections=None):
    """|a cos| + |b sin| of each output of rotate_rows: what an fp32 evaluation's error is relative to."""
    d = x.shape[-1]
    inv = inv_freq(d, theta)
    pos = np.asarray(positions, dtype=np.float64)
    phi = np.outer(pos, inv) if sections is None else pos[np.repeat(np.arange(3), sections)].T * inv
    c, s = np.abs(np.cos(phi))[:, None], np.abs(np.sin(phi))[:, None]
    a, b = np.abs(x[..., : d // 2]), np.abs(x[..., d // 2:])
    return np.concatenate([a * c + b * s, b * c + a * s], axis=-1)


def append_q8(values, scale, rows, table, first: int):
    """Rows [n][heads][d] of one sequence into the 8-bit cache, at positions
    first .. first + n - 1: values [pages][16][heads][d] and scale [pages][heads]
    (fp64) are changed in place."""
    n, heads, _ = rows.shape
    at = 0
    while at < n:
        page, slot = int(table[(first + at) // PAGE]), (first + at) % PAGE
        m = min(PAGE - slot, n - at)
        for h in range(heads):
            new = rows[at:at + m, h]
            s = q8_scale(new)
            if slot:
                s = max(s, scale[page, h])
                values[page, :slot, h] = e4m3_round(values[page, :slot, h] * (scale[page, h] / s))
            values[page, slot:slot + m, h] = e4m3_round(new / s)
            scale[page, h] = s
        at += m


def attend_rows(q, k, v, n_kv_heads: int, scale: float):
    """Causal attention of the last len(q) tokens: q [rows][n_q_heads][d], k, v
    [tokens][n_kv_heads][d].  Returns (out, log-sum-exp, sum_t p_t |v_t|)."""
    rows, hq, d = q.shape
    tokens, g = k.shape[0], hq // n_kv_heads
    out, mag = np.zeros((rows, hq, d)), np.zeros((rows, hq, d))
    lse = np.full((rows, hq), -np.inf)
    for i in range(rows):
        t = tokens - rows + i + 1
        for j in range(hq):
            s = scale * (k[:t, j // g] @ q[i, j])
            m = s.max()
            p = np.exp(s - m)
            lse[i, j] = m + np.log(p.sum())
            out[i, j] = (p / p.sum()) @ v[:t, j // g]
            mag[i, j] = (p / p.sum()) @ np.abs(v[:t, j // g])
    return out, lse, mag
