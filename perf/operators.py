"""The serving operators around a reused KV cache, as measurable cases.

Four operators carry a sequence on after its chunks were relocated into a paged cache of
16-token pages:

  append     the new rows of q, k, v of one layer: an RMS norm of each query and key head
             (optional), the position rotation (rotate-half RoPE or M-RoPE), q returned,
             k and v written into their slots of the paged bf16 cache
  append_q8  the same into a cache of e4m3 values with one fp32 scale for each (page, head)
  pack_q8    the pages of a bf16 chunk (one that was just relocated) into that 8-bit cache
  attend_q8  attention of the new rows over the 8-bit cache, causal, one row a sequence
             (decode), a few (draft verification) or many (a prompt behind reused chunks)

The 8-bit format: a block is the 16 tokens x head_dim values of one (page, head); it stands
for e4m3 value x scale with scale = 2^ceil(log2(amax / 448)), at least 2^-126, amax over the
block's finite values; what is not finite is stored as NaN.  A block that rows are appended
to keeps the larger of its scale and the new rows' one, its earlier rows being rounded again
under the new scale; a block whose first slot is written starts afresh.

`own` chooses between the plain form (elementary torch operations in 32 bits) and the
library's calls.  Both take the state that prepare() makes and write its buffers.
"""
import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False   # the plain products are 32-bit ones

own = False
PAGE = 16
EMIN = -126
SECTIONS = (16, 24, 24)   # M-RoPE frequency pairs per (t, h, w), head_dim 128


# --- the cases -----------------------------------------------------------------------
def listed():
    gqa = {"hq": 28, "hkv": 4, "d": 128, "theta": 1e6}
    mha = {"hq": 32, "hkv": 32, "d": 128, "theta": 1e4}
    return [
        # one decoded token of each of 16 sequences: the smallest append, all latency
        {"name": "append_decode", "op": "append", **gqa, "n": 16, "ctx_lo": 15, "ctx_hi": 4000,
         "rows_lo": 1, "rows_hi": 1, "norm": False, "mrope": False},
        # prompts with images behind reused chunks, ragged, query/key norms and M-RoPE
        {"name": "append_prompt", "op": "append", **gqa, "n": 8, "ctx_lo": 1, "ctx_hi": 1000,
         "rows_lo": 300, "rows_hi": 2500, "norm": True, "mrope": True},
        # one decoded token of each of 64 sequences into the 8-bit cache
        {"name": "append_q8_decode", "op": "append_q8", **gqa, "n": 64, "ctx_lo": 7, "ctx_hi": 2000,
         "rows_lo": 1, "rows_hi": 1, "norm": True, "mrope": False},
        # long prompts of a multi-head model into the 8-bit cache
        {"name": "append_q8_prompt", "op": "append_q8", **mha, "n": 4, "ctx_lo": 5, "ctx_hi": 700,
         "rows_lo": 501, "rows_hi": 3500, "norm": False, "mrope": False},
        # a relocated chunk of 4096 tokens, all 28 layers, into the 8-bit cache
        {"name": "pack_q8_chunk", "op": "pack_q8", "layers": 28, "tokens": 4096, "hkv": 4, "d": 128},
        # a short ragged chunk of two layers: launch latency and an open last page
        {"name": "pack_q8_short", "op": "pack_q8", "layers": 2, "tokens": 777, "hkv": 8, "d": 64},
        # one sequence, one token, a thousand cached: the smallest attention call
        {"name": "attend_one", "op": "attend_q8", **gqa, "n": 1, "ctx_lo": 999, "ctx_hi": 999,
         "rows_lo": 1, "rows_hi": 1},
        # the ordinary decode step: 16 sequences, each over 4 reused chunks of 4096 tokens
        {"name": "attend_decode", "op": "attend_q8", **gqa, "n": 16, "ctx_lo": 16383, "ctx_hi": 16383,
         "rows_lo": 1, "rows_hi": 1},
        # decode of a multi-head model over very uneven contexts
        {"name": "attend_ragged_mha", "op": "attend_q8", **mha, "n": 24, "ctx_lo": 37, "ctx_hi": 16000,
         "rows_lo": 1, "rows_hi": 1},
        # verification of four drafted tokens, head_dim 64
        {"name": "attend_verify", "op": "attend_q8", "hq": 32, "hkv": 8, "d": 64, "theta": 1e6, "n": 32,
         "ctx_lo": 900, "ctx_hi": 9000, "rows_lo": 4, "rows_hi": 4},
        # questions of different lengths behind reused chunks
        {"name": "attend_questions", "op": "attend_q8", **gqa, "n": 6, "ctx_lo": 500, "ctx_hi": 12000,
         "rows_lo": 37, "rows_hi": 900},
        # a long prompt behind a long reused context: the largest, all tensor-core work
        {"name": "attend_prompt", "op": "attend_q8", **gqa, "n": 1, "ctx_lo": 12345, "ctx_hi": 12345,
         "rows_lo": 4096, "rows_hi": 4096},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["append", "append_q8", "pack_q8", "attend_q8", "attend_q8"])
    if op == "pack_q8":
        hkv, d = rng.choice([1, 2, 3, 4, 8, 32]), rng.choice([64, 128])
        tokens = _log(rng, 5, 6000)
        layers = max(1, min(_log(rng, 1, 32), 28 * 4096 * 512 // (tokens * hkv * d)))
        return {"op": op, "layers": layers, "tokens": tokens, "hkv": hkv, "d": d}
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 4, 5, 7, 8, 16])
    c = {"op": op, "hq": hkv * g, "hkv": hkv, "d": d, "theta": rng.choice([1e4, 1e6])}
    kind = rng.choice(["decode", "decode", "verify", "prompt"])
    if kind == "decode":
        n, rows = _log(rng, 1, 64), (1, 1)
    elif kind == "verify":
        n, rows = _log(rng, 1, 32), (lambda r: (r, r))(rng.randint(2, 6))
    else:
        n = _log(rng, 1, 6)
        hi = _log(rng, 20, 1500)
        rows = (max(1, hi // rng.randint(1, 20)), hi)
    most = 16000 if op == "attend_q8" else 2000
    hi = _log(rng, 1, most)
    if op == "attend_q8":   # cached bytes and score terms stay below the largest listed cases'
        hi = max(1, min(hi, 16 * 16384 * 512 // (n * hkv * d), 28 * 4096 * 8192 // (n * hkv * g * rows[1])))
    c.update({"n": n, "ctx_lo": max(1, hi // rng.randint(1, 40)), "ctx_hi": hi, "rows_lo": rows[0], "rows_hi": rows[1]})
    if op != "attend_q8":
        c.update({"norm": rng.random() < 0.5, "mrope": d == 128 and rng.random() < 0.4})
    return c


def _spread(n, lo, hi, step):
    """n whole numbers from hi down to lo, evenly over their logarithm, in a mixed order."""
    v = [int(round(hi * (lo / hi) ** (i / max(1, n - 1)))) for i in range(n)]
    while math.gcd(step, n) != 1:
        step += 1
    return [v[(i * step) % n] for i in range(n)]


def _shape(c):
    """Cached tokens before the call and new rows, for each sequence."""
    return _spread(c["n"], c["ctx_lo"], c["ctx_hi"], 5), _spread(c["n"], c["rows_lo"], c["rows_hi"], 3)


def work(c):
    if c["op"] == "pack_q8":
        n = 2 * c["layers"] * c["tokens"] * c["hkv"] * c["d"]
        return {"bytes": 3 * n + 4 * n / (PAGE * c["d"]), "flops": 0}
    ctx, rows = _shape(c)
    n, kv = sum(rows), c["hkv"] * c["d"]
    q = 2 * n * c["hq"] * c["d"]
    if c["op"] == "append":
        return {"bytes": 2 * q + 8 * n * kv, "flops": 0}
    if c["op"] == "append_q8":
        return {"bytes": 2 * q + 6 * n * kv + 8 * n * c["hkv"] / PAGE, "flops": 0}
    tokens = sum(a + b for a, b in zip(ctx, rows))
    pairs = sum(a * b + b * (b + 1) // 2 for a, b in zip(ctx, rows))
    return {"bytes": 2 * tokens * kv * (1 + 4 / (PAGE * c["d"])) + 2 * q + 4 * n * c["hq"],
            "flops": 4 * pairs * c["hq"] * c["d"]}


# --- what a program has in hand before the call -----------------------------------------
def _rows(gen, *shape):
    """Rows as a projection gives them: N(0, 1) with a lognormal(0, 0.5) size for each feature, bf16."""
    size = torch.exp(0.5 * torch.randn(shape[-2:], generator=gen, device="cuda"))
    return (torch.randn(shape, generator=gen, device="cuda") * size).to(torch.bfloat16)


def _blocks(gen, pages, hkv, d):
    """A pool of 8-bit blocks as earlier calls left it, and its scales."""
    x = _rows(gen, pages, PAGE, hkv, d)
    e = _exponent(x.abs().amax(dim=(1, 3)).float())
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return (x.float() / scale[:, None, :, None]).to(torch.float8_e4m3fn), scale


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}
    hkv, d = c["hkv"], c["d"]
    if c["op"] == "pack_q8":
        pages = -(-c["tokens"] // PAGE)
        total = pages + 3
        src = [_rows(gen, c["layers"], total, PAGE, hkv, d) for _ in range(2)]
        pool = [torch.zeros((c["layers"], total, PAGE, hkv, d), dtype=torch.uint8, **dev).view(torch.float8_e4m3fn)
                for _ in range(2)]
        scale = [torch.zeros((c["layers"], total, hkv), dtype=torch.float32, **dev) for _ in range(2)]
        table = [torch.randperm(total, generator=gen, **dev)[:pages].to(torch.int32) for _ in range(2)]
        return {"c": c, "src": src, "pool": pool, "scale": scale, "src_table": table[0], "table": table[1],
                "pages": total, "kept": {}}
    ctx, rows = _shape(c)
    n, total_rows = c["n"], sum(rows)
    need = [-(-(a + b) // PAGE) for a, b in zip(ctx, rows)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=gen, **dev).to(torch.int32)
    starts = torch.tensor([sum(need[:i]) for i in range(n)], **dev)
    col = torch.arange(max(need), **dev)
    table = torch.where(col[None] < torch.tensor(need, **dev)[:, None],
                        order[(starts[:, None] + col[None]).clamp(max=pages - 1)], 0).to(torch.int32).contiguous()
    s = {"c": c, "table": table, "pages": pages, "n_rows": total_rows, "max_rows": max(rows), "kept": {},
         "seq_lens": torch.tensor([a + b for a, b in zip(ctx, rows)], dtype=torch.int32, **dev),
         "row_start": torch.tensor([sum(rows[:i]) for i in range(n + 1)], dtype=torch.int32, **dev),
         "seq_of": torch.repeat_interleave(torch.arange(n, **dev), torch.tensor(rows, **dev)),
         "one_each": max(rows) == 1}
    s["row_in"] = torch.arange(total_rows, **dev) - s["row_start"][s["seq_of"]]
    s["pos"] = (s["seq_lens"] - s["row_start"].diff())[s["seq_of"]] + s["row_in"]
    if c["op"] == "attend_q8":
        # queries as a trained model's: scores spread by about two units
        s["q"] = (2 * _rows(gen, total_rows, c["hq"], d).float() / 1.6).to(torch.bfloat16)
        s["k_pool"], s["k_scale"] = _blocks(gen, pages, hkv, d)
        s["v_pool"], s["v_scale"] = _blocks(gen, pages, hkv, d)
        s["out"] = torch.empty((total_rows, c["hq"], d), dtype=torch.bfloat16, **dev)
        s["lse"] = torch.empty((total_rows, c["hq"]), dtype=torch.float32, **dev)
        return s
    # the rows of a fused projection, [q | k | v] of each token
    s["qkv"] = _rows(gen, total_rows, c["hq"] + 2 * hkv, d)
    s["q_out"] = torch.empty((total_rows, c["hq"], d), dtype=torch.bfloat16, **dev)
    s["w"] = [(1 + 0.2 * torch.randn(d, generator=gen, **dev)).to(torch.bfloat16) for _ in range(2)] if c["norm"] else [None, None]
    s["positions"] = None
    if c["mrope"]:   # image tokens: a time index, rows and columns of a grid
        at = s["pos"]
        s["positions"] = torch.stack([at // 64, at // 64 + at % 64 // 8, at // 64 + at % 8]).to(torch.int32)
    if c["op"] == "append":
        s["pool"] = [_rows(gen, pages, PAGE, hkv, d) for _ in range(2)]
    else:
        s["pool"], s["scale"] = map(list, zip(*[_blocks(gen, pages, hkv, d) for _ in range(2)]))
    return s


# --- the plain form -----------------------------------------------------------------
def _exponent(amax):
    """The least e >= EMIN with amax <= 448 2^e."""
    m, e = torch.frexp(amax)
    return torch.where(amax > 0, e - 9 + (m > 0.875).to(e.dtype), EMIN).clamp(min=EMIN)


def _scale_of(x, dims):
    amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(dim=dims)
    return torch.ldexp(torch.ones_like(amax), _exponent(amax))


def _to_q8(x):
    return torch.where(torch.isfinite(x), x, float("nan")).to(torch.float8_e4m3fn)


def _rotated(s):
    """The new rows in 32 bits: q and k normed and rotated, v as it is."""
    c = s["c"]
    q, k, v = s["qkv"].float().split([c["hq"], c["hkv"], c["hkv"]], dim=1)
    if c["norm"]:
        q, k = ((x * torch.rsqrt((x * x).mean(-1, keepdim=True) + 1e-6)) * w.float() for x, w in ((q, s["w"][0]), (k, s["w"][1])))
    half = c["d"] // 2
    pair = torch.arange(half, device="cuda", dtype=torch.float64)
    inv = c["theta"] ** (-pair / half)
    if c["mrope"]:
        sec = (pair >= SECTIONS[0]).long() + (pair >= SECTIONS[0] + SECTIONS[1]).long()
        phi = s["positions"].double()[sec].T * inv
    else:
        phi = s["pos"].double()[:, None] * inv
    cos, sin = torch.cos(phi).float()[:, None], torch.sin(phi).float()[:, None]
    turn = lambda x: torch.cat([x[..., :half] * cos - x[..., half:] * sin, x[..., half:] * cos + x[..., :half] * sin], -1)  # noqa: E731
    return turn(q), turn(k), v


def _append(s):
    q, k, v = _rotated(s)
    page, slot = s["table"][s["seq_of"], s["pos"] // PAGE].long(), s["pos"] % PAGE
    for pool, x in zip(s["pool"], (k, v)):
        pool[page, slot] = x.to(torch.bfloat16)
    return {"q": q.to(torch.bfloat16), "k": s["pool"][0], "v": s["pool"][1]}


def _append_q8(s):
    q, k, v = _rotated(s)
    page, slot = s["table"][s["seq_of"], s["pos"] // PAGE].long(), s["pos"] % PAGE
    at = s["pos"][s["row_start"][:-1].long()]                       # each sequence's first new position
    first = s["table"].gather(1, (at // PAGE)[:, None].long())[:, 0].long()   # the one page that may hold earlier rows
    earlier = torch.arange(PAGE, device="cuda")[None] < (at % PAGE)[:, None]
    for pool, scale, x in zip(s["pool"], s["scale"], (k, v)):
        amax = torch.where(torch.isfinite(x), x.abs(), 0.0).amax(-1)
        most = torch.zeros_like(scale).scatter_reduce(0, page[:, None].expand_as(amax), amax, "amax")
        new = torch.ldexp(torch.ones_like(most), _exponent(most))
        old = scale[first]
        kept = torch.maximum(old, new[first]) * (at % PAGE > 0)[:, None]
        new[first] = torch.maximum(new[first], kept)
        ratio = (old / new[first])[:, None, :, None]
        block = pool[first]
        again = torch.where(earlier[:, :, None, None], block.float() * ratio, block.float()).to(torch.float8_e4m3fn)
        raw = pool.view(torch.uint8)
        raw[first] = again.view(torch.uint8)
        raw[page, slot] = _to_q8(x / new[page][..., None]).view(torch.uint8)
        scale[page] = new[page]
    return {"q": q.to(torch.bfloat16), "k": s["pool"][0], "v": s["pool"][1], "k_scale": s["scale"][0], "v_scale": s["scale"][1]}


def _pack_q8(s):
    c = s["c"]
    pages = -(-c["tokens"] // PAGE)
    held = torch.arange(pages * PAGE, device="cuda").view(pages, PAGE)[None, :, :, None, None] < c["tokens"]
    for src, pool, scale in zip(s["src"], s["pool"], s["scale"]):
        x = torch.where(held, src[:, s["src_table"].long()].float(), 0.0)
        e = _scale_of(x, (2, 4))
        pool.view(torch.uint8)[:, s["table"].long()] = _to_q8(x / e[:, :, None, :, None]).view(torch.uint8)
        scale[:, s["table"].long()] = e
    return {"k": s["pool"][0], "v": s["pool"][1], "k_scale": s["scale"][0], "v_scale": s["scale"][1]}


def _attend_q8(s):
    c, n, hkv, d = s["c"], s["c"]["n"], s["c"]["hkv"], s["c"]["d"]
    g, most, table = c["hq"] // hkv, s["max_rows"], s["table"].long()
    length, count = s["seq_lens"].long(), s["row_start"].diff().long()
    at = torch.arange(table.shape[1] * PAGE, device="cuda")
    r = torch.arange(most, device="cuda")
    row = (s["row_start"][:-1, None] + r[None]).clamp(max=s["n_rows"] - 1).long()
    pos = (length - count)[:, None] + r[None]                                             # [n, rows]
    seen = (at[None, None] <= pos[..., None]) & (at[None, None] < length[:, None, None])  # [n, rows, tokens]
    seen = seen[:, None, :, None, :].expand(n, hkv, most, g, -1).reshape(n, hkv, most * g, -1)
    values = lambda pool, scale: (pool[table].float() * scale[table][:, :, None, :, None]).view(n, -1, hkv, d)  # noqa: E731
    q = s["q"][row].float().view(n, most, hkv, g, d).transpose(1, 2).reshape(n, hkv, most * g, d)
    x = q @ values(s["k_pool"], s["k_scale"]).permute(0, 2, 3, 1) * d ** -0.5
    x = torch.where(seen, x, float("-inf"))
    top = x.amax(-1, keepdim=True)
    top = torch.where(torch.isinf(top), 0.0, top)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    v = torch.where((at[None] < length[:, None])[..., None, None], values(s["v_pool"], s["v_scale"]), 0.0)
    o = p @ v.transpose(1, 2) / torch.where(total > 0, total, 1.0)
    lse = top + torch.log(total)
    back = lambda y: y.view(n, hkv, most, g, -1).permute(0, 2, 1, 3, 4)[s["seq_of"], s["row_in"]].reshape(s["n_rows"], c["hq"], -1)  # noqa: E731
    return {"out": back(o).to(torch.bfloat16), "lse": back(lse)[..., 0]}


# --- the library's calls ---------------------------------------------------------------
def _seqs(s, kvrp):
    if "seqs" not in s["kept"]:
        s["kept"]["seqs"] = kvrp.Seqs(seq_lens=s["seq_lens"], block_tables=s["table"], num_pages=s["pages"],
                                      n_rows=s["n_rows"], row_start=None if s["one_each"] else s["row_start"],
                                      max_rows=s["max_rows"])
    return s["kept"]["seqs"]


def _own(s):
    import position_invariant_kv_gb300 as kvrp
    c = s["c"]
    if c["op"] == "pack_q8":
        kvrp.kv_pack_q8(s["src"][0], s["src"][1], n_layers=c["layers"], n_tokens=c["tokens"], n_kv_heads=c["hkv"],
                        head_dim=c["d"], src_table=s["src_table"], src_pages=s["pages"],
                        k_pool=s["pool"][0], v_pool=s["pool"][1], k_scale=s["scale"][0], v_scale=s["scale"][1],
                        block_table=s["table"], num_pages=s["pages"])
        return {"k": s["pool"][0], "v": s["pool"][1], "k_scale": s["scale"][0], "v_scale": s["scale"][1]}
    if c["op"] == "attend_q8":
        if "ws" not in s["kept"]:
            size = kvrp.kv_attend_q8_workspace_size(c["hq"], c["hkv"], c["d"], s["max_rows"])
            s["kept"]["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
        kvrp.kv_attend_q8(s["q"], _seqs(s, kvrp), n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=c["d"],
                          softmax_scale=c["d"] ** -0.5, k_pool=s["k_pool"], v_pool=s["v_pool"], k_scale=s["k_scale"],
                          v_scale=s["v_scale"], out=s["out"], lse=s["lse"], workspace=s["kept"]["ws"])
        return {"out": s["out"], "lse": s["lse"]}
    q, k, v = s["qkv"][:, :c["hq"]], s["qkv"][:, c["hq"]:c["hq"] + c["hkv"]], s["qkv"][:, c["hq"] + c["hkv"]:]
    width = (c["hq"] + 2 * c["hkv"]) * c["d"]
    same = dict(n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=c["d"], rope_theta=c["theta"], q_out=s["q_out"],
                q_stride=width, k_stride=width, v_stride=width, q_norm=s["w"][0], k_norm=s["w"][1], norm_eps=1e-6,
                positions=s["positions"], mrope_section=SECTIONS if c["mrope"] else None,
                k_pool=s["pool"][0], v_pool=s["pool"][1])
    if c["op"] == "append":
        kvrp.kv_append(q, k, v, _seqs(s, kvrp), **same)
        return {"q": s["q_out"], "k": s["pool"][0], "v": s["pool"][1]}
    kvrp.kv_append_q8(q, k, v, _seqs(s, kvrp), k_scale=s["scale"][0], v_scale=s["scale"][1], **same)
    return {"q": s["q_out"], "k": s["pool"][0], "v": s["pool"][1], "k_scale": s["scale"][0], "v_scale": s["scale"][1]}


def run(s):
    if own:
        return _own(s)
    return {"append": _append, "append_q8": _append_q8, "pack_q8": _pack_q8, "attend_q8": _attend_q8}[s["c"]["op"]](s)


# --- the definitions in 64 bits, written apart from the plain form -------------------------
def _e4m3(x):
    """x rounded to the nearest e4m3 value, ties to even (|x| <= 448 or NaN)."""
    a = x.abs()
    e = torch.floor(torch.log2(torch.where(a > 0, a, 1.0))).clamp(min=-6)
    e = torch.where(2.0 ** (e + 1) <= a, e + 1, e)   # log2's rounding next to a power of two
    e = torch.where(2.0 ** e > a, e - 1, e).clamp(min=-6)
    step = 2.0 ** (e - 3)
    return torch.round(x / step) * step


def _block_scale(x, heads_dim):
    a = torch.where(torch.isfinite(x), x.abs(), 0.0)
    a = a.amax(dim=[i for i in range(x.dim()) if i != heads_dim])
    e = torch.ceil(torch.log2(torch.where(a > 0, a, 1.0) / 448))
    e = torch.where(448 * 2.0 ** (e - 1) >= a, e - 1, e)
    e = torch.where(448 * 2.0 ** e < a, e + 1, e)
    return 2.0 ** torch.where(a > 0, e, float(EMIN)).clamp(min=float(EMIN))


def exact(c, seed):
    s = prepare(c, seed)
    if c["op"] == "pack_q8":
        got = {}
        src_t, dst_t = s["src_table"].tolist(), s["table"].tolist()
        for name, src, pool, scale in zip("kv", s["src"], s["pool"], s["scale"]):
            rows, factor = pool.double(), scale.double()
            for i, (a, b) in enumerate(zip(src_t, dst_t)):
                x = src[:, a].double()
                x[:, max(0, c["tokens"] - i * PAGE):] = 0
                f = torch.stack([_block_scale(y, 1) for y in x]) if c["layers"] < 4 else _layers_scale(x)
                rows[:, b], factor[:, b] = _e4m3(x / f[:, None, :, None]), f
            got[name], got[name + "_scale"] = rows, factor
        return got
    if c["op"] == "attend_q8":
        return _exact_attend(c, s)
    q, k, v = s["qkv"].double().split([c["hq"], c["hkv"], c["hkv"]], dim=1)
    if c["norm"]:
        q, k = (x / torch.sqrt((x ** 2).sum(-1, keepdim=True) / c["d"] + 1e-6) * w.double() for x, w in ((q, s["w"][0]), (k, s["w"][1])))
    ang = []
    for i in range(c["d"] // 2):
        p = s["pos"].double()
        if c["mrope"]:
            p = s["positions"][0 if i < 16 else 1 if i < 40 else 2].double()
        ang.append(p * math.pow(c["theta"], -2.0 * i / c["d"]))
    unit = torch.polar(torch.ones_like(ang[0])[:, None], torch.stack(ang, -1))[:, None]
    turned = []
    for x in (q, k):
        z = torch.complex(x[..., :c["d"] // 2].contiguous(), x[..., c["d"] // 2:].contiguous()) * unit
        turned.append(torch.cat([z.real, z.imag], -1))
    q, k = turned
    ctx, rows = _shape(c)
    table, got, start = s["table"].tolist(), {"q": q}, 0
    pools = [p.double() for p in s["pool"]]
    scales = [f.double() for f in s["scale"]] if c["op"] == "append_q8" else None
    for i in range(c["n"]):
        at, end = ctx[i], ctx[i] + rows[i]
        while at < end:
            stop = min(end, (at // PAGE + 1) * PAGE)
            page, a, b = table[i][at // PAGE], at % PAGE, at % PAGE + stop - at
            for j, x in enumerate((k, v)):
                new = x[start:start + stop - at]
                if scales is None:
                    pools[j][page, a:b] = new
                    continue
                f = _block_scale(new, 1)
                if a:
                    f = torch.maximum(f, scales[j][page])
                    pools[j][page, :a] = _e4m3(pools[j][page, :a] * (scales[j][page] / f)[None, :, None])
                pools[j][page, a:b] = _e4m3(new / f[None, :, None])
                scales[j][page] = f
            start += stop - at
            at = stop
    got["k"], got["v"] = pools
    if scales is not None:
        got["k_scale"], got["v_scale"] = scales
    return got


def _layers_scale(x):
    """_block_scale of each layer of [layers, 16, heads, d]."""
    y = x.permute(0, 2, 1, 3).reshape(1, x.shape[0] * x.shape[2], -1)
    return _block_scale(y, 1).view(x.shape[0], x.shape[2])


def _exact_attend(c, s):
    ctx, rows = _shape(c)
    hkv, g, d = c["hkv"], c["hq"] // c["hkv"], c["d"]
    out = torch.zeros((s["n_rows"], c["hq"], d), dtype=torch.float64, device="cuda")
    lse = torch.zeros((s["n_rows"], c["hq"]), dtype=torch.float64, device="cuda")
    start = 0
    for i in range(c["n"]):
        t = ctx[i] + rows[i]
        pages = s["table"][i, :-(-t // PAGE)].long()
        later = torch.arange(t, device="cuda")[None] > torch.arange(ctx[i], t, device="cuda")[:, None]
        for h in range(hkv):
            k, v = ((s[n + "_pool"][pages][:, :, h].double() * s[n + "_scale"][pages][:, h, None, None].double()).reshape(-1, d)[:t]
                    for n in "kv")
            for j in range(h * g, (h + 1) * g):
                x = (s["q"][start:start + rows[i], j].double() / math.sqrt(d)) @ k.T
                x.masked_fill_(later, -math.inf)
                lse[start:start + rows[i], j] = torch.logsumexp(x, -1)
                out[start:start + rows[i], j] = torch.softmax(x, -1) @ v
        start += rows[i]
    return {"out": out, "lse": lse}
