"""Decode steps with drafted tokens behind one long shared context, as measurable cases.

Three operators carry a batch of sequences through such a step over the paged 8-bit cache
of 16-token pages:

  step_tables    the batch of the next step, built on the device from each sequence's kept
                 tokens and new rows: row starts, lengths, block tables (pages taken from a
                 ring of free ones and given back to it), positions and slots of the rows
  attend_shared  attention of the new rows over the 8-bit cache where all sequences begin
                 with the same tokens: the shared pages are read once for the whole batch
  verify         drafted tokens kept or not against the target's probabilities, from given
                 random numbers, and the token that follows the last one kept

The ring of free pages: ring[(head + i) % size], i < count, in the order in which they are
taken; what a call gives back goes behind them and can be taken from the next call on.

The draw of a token: weights w are whole numbers, the probability times 2^40 rounded down
(of a rejected draft's row the positive part of target minus draft); the token is the first
one at which their running sum passes floor(floor(2^32 u) * sum / 2^32).

`own` chooses between the plain form (elementary torch operations in 32 bits, whole numbers
in 64) and the library's calls.  Both take the state that prepare() makes.
"""
import math

import torch

if torch.cuda.is_available():
    torch.backends.cuda.matmul.allow_tf32 = False   # the plain products are 32-bit ones

own = False
PAGE = 16
EMIN = -126
HOLD = 0.75   # about the share of drawn drafts that the target keeps


# --- the cases -----------------------------------------------------------------------
def listed():
    gqa = {"hq": 28, "hkv": 4, "d": 128}
    return [
        # 64 running sequences, 4 drafts each and the token before them: all latency
        {"name": "tables_decode", "op": "step_tables", "n": 64, "ctx_lo": 40, "ctx_hi": 4000, "rows_lo": 5, "rows_hi": 5,
         "prefix": 0, "fresh": 0, "done": 0},
        # new prompts of very different lengths behind a shared context, some places just given up
        {"name": "tables_prompts", "op": "step_tables", "n": 48, "ctx_lo": 1, "ctx_hi": 900, "rows_lo": 37, "rows_hi": 6000,
         "prefix": 1024, "fresh": 2, "done": 7},
        # three users on a short shared context: the smallest attention call
        {"name": "attend_small", "op": "attend_shared", **gqa, "n": 3, "prefix": 1008, "ctx_lo": 1, "ctx_hi": 90, "rows": 1},
        # the ordinary decode step: 64 sequences over 4 reused chunks of 4096 tokens and their own turns
        {"name": "attend_decode", "op": "attend_shared", **gqa, "n": 64, "prefix": 16384, "ctx_lo": 30, "ctx_hi": 1500, "rows": 1},
        # a multi-head model
        {"name": "attend_mha", "op": "attend_shared", "hq": 32, "hkv": 32, "d": 128, "n": 24, "prefix": 4144, "ctx_lo": 20,
         "ctx_hi": 700, "rows": 1},
        # three drafts and the token before them, head_dim 64
        {"name": "attend_verify", "op": "attend_shared", "hq": 32, "hkv": 8, "d": 64, "n": 32, "prefix": 9008, "ctx_lo": 10,
         "ctx_hi": 900, "rows": 4},
        # longer drafts over a long document: more (row, head) pairs a sequence than a decode tile holds
        {"name": "attend_drafts", "op": "attend_shared", **gqa, "n": 16, "prefix": 65536, "ctx_lo": 40, "ctx_hi": 2000, "rows": 5},
        # many users of a book: the largest, the tensor cores' work
        {"name": "attend_large", "op": "attend_shared", **gqa, "n": 96, "prefix": 100000, "ctx_lo": 100, "ctx_hi": 3000, "rows": 1},
        # one user, drafts looked up in the prompt (no draft distribution): latency
        {"name": "verify_one", "op": "verify", "n": 1, "vocab": 32000, "rows_lo": 5, "rows_hi": 5, "bf16": False, "draft": False},
        # the ordinary step of a batch, vocabulary of an odd size
        {"name": "verify_batch", "op": "verify", "n": 64, "vocab": 130003, "rows_lo": 5, "rows_hi": 5, "bf16": False, "draft": True},
        # drafts of different lengths, probabilities in bf16
        {"name": "verify_ragged", "op": "verify", "n": 37, "vocab": 50021, "rows_lo": 1, "rows_hi": 8, "bf16": True, "draft": True},
        # a large batch and vocabulary: memory
        {"name": "verify_large", "op": "verify", "n": 256, "vocab": 262144, "rows_lo": 4, "rows_hi": 4, "bf16": False, "draft": True},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["step_tables", "attend_shared", "attend_shared", "verify"])
    if op == "step_tables":
        decode = rng.random() < 0.6
        n = _log(rng, 1, 3000 if decode else 64)
        rows = rng.randint(1, 8) if decode else _log(rng, 10, 6000)
        ctx = _log(rng, 1, 4000)
        return {"op": op, "n": n, "ctx_lo": max(1, ctx // rng.randint(1, 40)), "ctx_hi": ctx,
                "rows_lo": max(1, rows // rng.randint(1, 20)), "rows_hi": rows, "prefix": rng.choice([0, _log(rng, 1, 1024)]),
                "fresh": rng.choice([0, 2, 5]), "done": rng.choice([0, 3, 7])}
    if op == "verify":
        vocab = _log(rng, 500, 262144)
        n = min(_log(rng, 1, 256), max(1, 256 * 262144 // vocab))
        rows = rng.randint(1, 8) if n * vocab < 128 * 262144 else rng.randint(1, 4)
        return {"op": op, "n": n, "vocab": vocab, "rows_lo": max(1, rows - rng.randint(0, 7)), "rows_hi": rows,
                "bf16": rng.random() < 0.4, "draft": rng.random() < 0.7}
    d = rng.choice([64, 128, 128])
    hkv = rng.choice([1, 2, 3, 4, 8])
    g = rng.choice([1, 2, 4, 5, 7, 8, 16])
    n, rows = _log(rng, 1, 96), rng.choice([1, 1, 1, rng.randint(2, 8)])
    ctx = min(_log(rng, 1, 3000), max(1, 96 * 1500 * 512 // (n * hkv * d)))
    prefix = min(_log(rng, 1, 65536), max(1, 96 * 100000 * 28 * 128 // (2 * n * rows * hkv * g * d)))
    return {"op": op, "hq": hkv * g, "hkv": hkv, "d": d, "n": n, "prefix": max(PAGE, prefix // PAGE * PAGE),
            "ctx_lo": max(1, ctx // rng.randint(1, 40)), "ctx_hi": ctx, "rows": rows}


def _spread(n, lo, hi, step):
    """n whole numbers from hi down to lo, evenly over their logarithm, in a mixed order."""
    v = [int(round(hi * (lo / hi) ** (i / max(1, n - 1)))) for i in range(n)]
    while math.gcd(step, n) != 1:
        step += 1
    return [v[(i * step) % n] for i in range(n)]


def _pages(tokens):
    return -(-tokens // PAGE)


def _batch(c):
    """step_tables: for each sequence its kept tokens, new rows and the pages that it holds."""
    ctx, rows = _spread(c["n"], c["ctx_lo"], c["ctx_hi"], 5), _spread(c["n"], c["rows_lo"], c["rows_hi"], 3)
    first, kept, new, held = c["prefix"] * PAGE, [], [], []
    for i in range(c["n"]):
        if c["done"] and i % c["done"] == 1:       # a sequence that has ended: its pages go back
            kept.append(0)
            new.append(0)
            held.append(_pages(first + ctx[i]))
        elif c["fresh"] and i % c["fresh"] == 0:   # one that begins, behind the shared pages
            kept.append(first)
            new.append(rows[i])
            held.append(0)
        else:                                      # one that goes on: some of its last rows were drafts not kept
            kept.append(first + ctx[i])
            new.append(rows[i])
            held.append(_pages(first + ctx[i] + i % 40))
    return kept, new, held


def work(c):
    if c["op"] == "step_tables":
        kept, new, held = _batch(c)
        need = [_pages(a + b) for a, b in zip(kept, new)]
        moved = sum(abs(a - b) for a, b in zip(need, held))
        return {"bytes": 4 * 6 * c["n"] + 8 * moved + 12 * sum(new), "flops": 0}
    if c["op"] == "verify":
        rows = _spread(c["n"], c["rows_lo"], c["rows_hi"], 3)
        read = sum(1 + (1 - HOLD ** (r - 1) if c["draft"] else 0) for r in rows)   # a kept row of drafts reads the target's only
        return {"bytes": read * c["vocab"] * (2 if c["bf16"] else 4) + 16 * sum(rows), "flops": 0}
    ctx = _spread(c["n"], c["ctx_lo"], c["ctx_hi"], 5)
    r, n = c["rows"], c["n"] * c["rows"]
    tokens = c["prefix"] + sum(ctx) + n
    pairs = n * c["prefix"] + sum(a * r + r * (r + 1) // 2 for a in ctx)
    return {"bytes": 2 * tokens * c["hkv"] * c["d"] * (1 + 4 / (PAGE * c["d"])) + 4 * n * c["hq"] * c["d"],
            "flops": 4 * pairs * c["hq"] * c["d"]}


# --- what a program has in hand before the call -----------------------------------------
def _rows(gen, *shape):
    """Rows as a projection gives them: N(0, 1) with a lognormal(0, 0.5) size for each feature, bf16."""
    size = torch.exp(0.5 * torch.randn(shape[-2:], generator=gen, device="cuda"))
    return (torch.randn(shape, generator=gen, device="cuda") * size).to(torch.bfloat16)


def _blocks(gen, pages, hkv, d):
    """A pool of 8-bit blocks as earlier calls left it, and its scales."""
    x = _rows(gen, pages, PAGE, hkv, d)
    m, e = torch.frexp(x.abs().amax(dim=(1, 3)).float())
    e = torch.where(m > 0, e - 9 + (m > 0.875).to(e.dtype), EMIN).clamp(min=EMIN)
    scale = torch.ldexp(torch.ones_like(e, dtype=torch.float32), e)
    return (x.float() / scale[:, None, :, None]).to(torch.float8_e4m3fn), scale


def _i32(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dev = {"device": "cuda"}
    n = c["n"]
    if c["op"] == "step_tables":
        kept, new, held = _batch(c)
        first, rows = c["prefix"], sum(new)
        stride = max(_pages(a + b) for a, b in zip(kept, new)) + 2
        stride = max([stride] + held)
        own_pages = [max(0, h - first) for h in held]
        taken = sum(max(0, _pages(a + b) - max(h, first)) for a, b, h in zip(kept, new, held) if a + b)
        pages = first + sum(own_pages) + taken + 5
        order = torch.randperm(pages, generator=gen, **dev).to(torch.int32)
        col = torch.arange(stride, **dev)
        start = first + _i32([sum(own_pages[:i]) for i in range(n)]).long()
        mine = order[(start[:, None] + (col - first)[None]).clamp(0, pages - 1)]
        table = torch.where(col[None] < first, order[col.clamp(max=pages - 1)][None], mine)
        table = torch.where(col[None] < _i32(held)[:, None], table, 0).contiguous()
        free = pages - first - sum(own_pages)
        head = int(torch.randint(0, pages, (1,), generator=torch.Generator().manual_seed(seed)))
        ring = torch.zeros(pages, dtype=torch.int32, **dev)
        ring[(head + torch.arange(free, **dev)) % pages] = order[first + sum(own_pages):]
        return {"c": c, "kept": _i32(kept), "new": _i32(new), "held": _i32(held), "table": table, "ring": ring, "pages": pages,
                "free": _i32([head, free]), "n_rows": rows, "max_rows": max(new), "prefix_table": order[:first].contiguous(),
                "prefix_len": _i32([first * PAGE]), "row_start": _i32([0] * (n + 1)), "seq_lens": _i32([0] * n),
                "held_out": _i32([0] * n), "free_out": _i32([0, 0]), "positions": torch.zeros(rows, dtype=torch.int32, **dev),
                "slots": torch.zeros(rows, dtype=torch.int64, **dev), "plan": {}}
    if c["op"] == "verify":
        count = _spread(n, c["rows_lo"], c["rows_hi"], 3)
        rows, vocab = sum(count), c["vocab"]
        kind = torch.bfloat16 if c["bf16"] else torch.float32
        target = torch.empty((rows, vocab), dtype=kind, **dev)
        draft = torch.empty((rows, vocab), dtype=kind, **dev) if c["draft"] else None
        starts = [sum(count[:i]) for i in range(n + 1)]
        tokens = torch.zeros(rows + 1, dtype=torch.int32, **dev)
        tokens[0] = vocab // 2
        for a in range(0, rows, 64):   # a model's next-token logits, a smaller model's near them, and what it drew
            logits = 2.5 * torch.randn((min(64, rows - a), vocab), generator=gen, **dev)
            some = torch.randint(0, vocab, (logits.shape[0], 1), generator=gen, **dev)   # one token stands out, more or less
            logits.scatter_(1, some, math.log(vocab) + 4 + 2 * torch.randn(some.shape, generator=gen, **dev))
            target[a:a + 64] = torch.softmax(logits, -1).to(kind)
            near = torch.softmax(logits + 0.75 * torch.randn(logits.shape, generator=gen, **dev), -1).to(kind)
            if c["draft"]:
                draft[a:a + 64] = near
            race = torch.empty(logits.shape, **dev).exponential_(generator=gen)
            # a looked-up draft is often the likeliest token
            drawn = (near.float() / race).argmax(-1) if c["draft"] else near.argmax(-1)
            tokens[a + 1:a + 1 + drawn.numel()] = drawn.to(torch.int32)   # drawn from row r, it is row r + 1's token
        return {"c": c, "target": target, "draft": draft, "tokens": tokens[:rows].contiguous(), "n_rows": rows,
                "max_rows": max(count), "row_start": _i32(starts), "seq_lens": _i32([r + 100 + i for i, r in enumerate(count)]),
                "table": _i32([[0] * 40] * n), "u_accept": torch.rand(rows, generator=gen, **dev),
                "u_sample": torch.rand(n, generator=gen, **dev), "out": torch.zeros(rows, dtype=torch.int32, **dev),
                "accepted": _i32([0] * n), "kept": _i32([0] * n), "plan": {}}
    ctx = _spread(n, c["ctx_lo"], c["ctx_hi"], 5)
    hkv, d, r, first = c["hkv"], c["d"], c["rows"], c["prefix"] // PAGE
    need = [_pages(a + r) for a in ctx]
    pages = first + sum(need) + 3
    order = torch.randperm(pages, generator=gen, **dev).to(torch.int32)
    start = first + _i32([sum(need[:i]) for i in range(n)]).long()
    col = torch.arange(first + max(need), **dev)
    mine = order[(start[:, None] + (col - first)[None]).clamp(0, pages - 1)]
    table = torch.where(col[None] < first, order[col.clamp(max=pages - 1)][None], mine)
    table = torch.where(col[None] < first + _i32(need)[:, None], table, 0).contiguous()
    s = {"c": c, "table": table, "pages": pages, "n_rows": n * r, "max_rows": r, "prefix_table": order[:first].contiguous(),
         "prefix_len": _i32([c["prefix"]]), "row_start": _i32([i * r for i in range(n + 1)]),
         "seq_lens": _i32([c["prefix"] + a + r for a in ctx]), "plan": {},
         # queries as a trained model's: scores spread by about two units
         "q": (2 * _rows(gen, n * r, c["hq"], d).float() / 1.6).to(torch.bfloat16),
         "out": torch.empty((n * r, c["hq"], d), dtype=torch.bfloat16, **dev)}
    s["k_pool"], s["k_scale"] = _blocks(gen, pages, hkv, d)
    s["v_pool"], s["v_scale"] = _blocks(gen, pages, hkv, d)
    return s


# --- the plain form -----------------------------------------------------------------
def _step_tables(s):
    n, first, pages = s["c"]["n"], s["c"]["prefix"], s["pages"]
    kept, new, held = s["kept"].long(), s["new"].long(), s["held"].long()
    head, count = s["free"][0].long(), s["free"][1].long()
    need = (kept + new + PAGE - 1) // PAGE
    takes = torch.where(need > 0, need - held.clamp(min=first), 0).clamp(min=0)
    upto = takes.cumsum(0)
    served = (takes == 0) | (upto <= count)
    ring = s["ring"]
    # table entries that are new: the shared pages of a sequence that begins, then pages taken
    at = torch.arange(s["table"].shape[1], device="cuda")[None]
    nth = (upto - takes)[:, None] + at - held.clamp(min=first)[:, None]
    shared = s["prefix_table"][at.clamp(max=first - 1)] if first else torch.zeros_like(at, dtype=torch.int32)
    fill = torch.where(at < first, shared, ring[(head + nth.clamp(min=0)) % pages])
    table = torch.where(served[:, None] & (at >= held[:, None]) & (at < need[:, None]), fill, s["table"])
    # pages given back go behind the free ones
    stay = torch.where(need > 0, need.clamp(min=first), first)
    back = torch.where(served, held - stay, 0).clamp(min=0)
    before = back.cumsum(0) - back
    place = torch.where((at >= stay[:, None]) & (at < held[:, None]) & served[:, None],
                        (head + count + before[:, None] + at - stay[:, None]) % pages, pages)
    more = torch.cat([ring, ring[:1]])
    more.scatter_(0, place.flatten(), s["table"].flatten())
    ring.copy_(more[:pages])
    s["table"].copy_(table)
    took = torch.where(served, takes, 0).sum()
    s["free_out"].copy_(torch.stack([(head + took) % pages, count - took + back.sum()]))
    s["held_out"].copy_(torch.where(served, need, held))
    s["row_start"][1:] = new.cumsum(0)
    s["seq_lens"].copy_(torch.where(served, kept + new, 0))
    row = torch.arange(s["n_rows"], device="cuda")
    of = torch.searchsorted(s["row_start"][1:].long(), row, right=True)
    pos = kept[of] + row - s["row_start"][of]
    s["positions"].copy_(torch.where(served[of], pos, 0))
    s["slots"].copy_(torch.where(served[of], table[of, pos // PAGE].long() * PAGE + pos % PAGE, -1))
    return _tables_out(s)


def _tables_out(s):
    return {k: s[k] for k in ("table", "ring", "free_out", "held_out", "row_start", "seq_lens", "positions", "slots")}


def _weights(x):
    """Probabilities as whole numbers of 2^-40."""
    return (x.double().nan_to_num(0.0).clamp(0.0, 1.0) * 2.0 ** 40).long()


def _verify(s):
    n, rows = s["c"]["n"], s["n_rows"]
    start, end = s["row_start"][:-1].long(), s["row_start"][1:].long()
    row = torch.arange(rows, device="cuda")
    last = (row[:, None] == (end - 1)[None]).any(-1)
    token = torch.where(last, 0, s["tokens"].long()[(row + 1).clamp(max=rows - 1)])
    p = s["target"].gather(1, token[:, None])[:, 0].double()
    q = s["draft"].gather(1, token[:, None])[:, 0].double() if s["draft"] is not None else torch.ones_like(p)
    stop = last | ~(s["u_accept"].double() * q < p)                # the first of a sequence is where its drafts end
    where = torch.where(stop, row, rows)
    at = torch.stack([where, row]).amin(0)                         # rows that stop; others count as past the end
    at = torch.where(stop, at, rows)
    first = torch.where(at[None] >= start[:, None], at[None], rows).amin(-1)
    ended = last[first]
    w = _weights(s["target"][first])
    gone = _weights(s["draft"][first]) if s["draft"] is not None else torch.zeros_like(w)
    if s["draft"] is None:   # a point at the drafted token
        gone.scatter_(1, token[first][:, None], 2 ** 40)
    rest = torch.where(ended[:, None], w, (w - gone).clamp(min=0))
    w = torch.where(rest.sum(-1, keepdim=True) > 0, rest, w)
    upto = w.cumsum(-1)
    total = upto[:, -1]
    u = (s["u_sample"].double() * 2.0 ** 32).long()
    high, low = total >> 20, total & (2 ** 20 - 1)                 # u * total / 2^32 in 64 bits
    t = (u * high >> 12) + (((u * high & 4095) << 20) + u * low >> 32)
    drawn = torch.searchsorted(upto, t[:, None], right=True)[:, 0]
    of = torch.searchsorted(end, row, right=True)
    s["out"].copy_(torch.where(row < first[of], token, torch.where(row == first[of], drawn[of], -1)))
    s["accepted"].copy_(first - start)
    s["kept"].copy_(s["seq_lens"] - (end - 1 - first))
    return {"out": s["out"], "accepted": s["accepted"], "kept": s["kept"]}


def _attend_shared(s):
    c = s["c"]
    n, hkv, d, r, first = c["n"], c["hkv"], c["d"], c["rows"], c["prefix"] // PAGE
    g = c["hq"] // hkv
    values = lambda pool, scale, t: pool[t].float() * scale[t][..., None, :, None]  # noqa: E731
    q = s["q"].float().view(n, r, hkv, g, d).permute(2, 0, 1, 3, 4) * d ** -0.5       # [hkv, n, r, g, d]
    t = s["prefix_table"].long()
    k = values(s["k_pool"], s["k_scale"], t).view(-1, hkv, d)
    x = (q.reshape(hkv, -1, d) @ k.permute(1, 2, 0)).view(hkv, n, r * g, -1)            # over the shared tokens
    t = s["table"][:, first:].long()
    k = values(s["k_pool"], s["k_scale"], t).view(n, -1, hkv, d)
    y = q.reshape(hkv, n, r * g, d) @ k.permute(2, 0, 3, 1)                             # over a sequence's own
    at = torch.arange(y.shape[-1], device="cuda")
    seen = s["seq_lens"].long()[:, None] - r + torch.arange(r, device="cuda")[None] + 1 - c["prefix"]
    seen = at[None, None] < seen.repeat_interleave(g, 1)[..., None]
    y = torch.where(seen[None], y, float("-inf"))
    top = torch.maximum(x.amax(-1, keepdim=True), y.amax(-1, keepdim=True))
    x, y = torch.exp(x - top), torch.exp(y - top)
    total = x.sum(-1, keepdim=True) + y.sum(-1, keepdim=True)
    v = values(s["v_pool"], s["v_scale"], s["prefix_table"].long()).view(-1, hkv, d)
    o = (x.view(hkv, n * r * g, -1) @ v.permute(1, 0, 2)).view(hkv, n, r * g, d)
    v = values(s["v_pool"], s["v_scale"], t).view(n, -1, hkv, d)
    o = (o + y @ v.permute(2, 0, 1, 3)) / total
    s["out"].copy_(o.view(hkv, n, r, g, d).permute(1, 2, 0, 3, 4).reshape(n * r, c["hq"], d))
    return {"out": s["out"]}


# --- the library's calls ---------------------------------------------------------------
def _own(s):
    import position_invariant_kv_gb300 as kvrp
    c, plan = s["c"], s["plan"]
    if "seqs" not in plan:
        plan["seqs"] = kvrp.Seqs(seq_lens=s["seq_lens"], block_tables=s["table"], num_pages=s.get("pages", 1),
                                 n_rows=s["n_rows"], row_start=s["row_start"], max_rows=s["max_rows"])
        if c.get("prefix"):
            plan["prefix"] = kvrp.Prefix(block_table=s["prefix_table"], length=s["prefix_len"])
    seqs = plan["seqs"]
    if c["op"] == "step_tables":
        kvrp.kv_step_tables(s["kept"], s["new"], seqs, held_pages=s["held"], held_out=s["held_out"], free_pages=s["ring"],
                            free_state=s["free"], free_state_out=s["free_out"], prefix=plan.get("prefix"),
                            positions=s["positions"], slots=s["slots"])
        return _tables_out(s)
    if c["op"] == "verify":
        kvrp.kv_verify_drafts(s["target"], seqs, vocab=c["vocab"], prob_type=kvrp.KVRP_BF16 if c["bf16"] else kvrp.KVRP_F32,
                              draft=s["draft"], tokens=s["tokens"], u_accept=s["u_accept"], u_sample=s["u_sample"],
                              out_tokens=s["out"], accepted=s["accepted"], kept_lens=s["kept"])
        return {"out": s["out"], "accepted": s["accepted"], "kept": s["kept"]}
    if "ws" not in plan:
        size = kvrp.kv_attend_shared_q8_workspace_size(c["hq"], c["hkv"], c["d"], s["max_rows"], s["n_rows"])
        plan["ws"] = torch.empty(size, dtype=torch.uint8, device="cuda")
    kvrp.kv_attend_shared_q8(s["q"], seqs, plan["prefix"], n_q_heads=c["hq"], n_kv_heads=c["hkv"], head_dim=c["d"],
                             softmax_scale=c["d"] ** -0.5, k_pool=s["k_pool"], v_pool=s["v_pool"], k_scale=s["k_scale"],
                             v_scale=s["v_scale"], out=s["out"], workspace=plan["ws"])
    return {"out": s["out"]}


def run(s):
    if own:
        return _own(s)
    return {"step_tables": _step_tables, "attend_shared": _attend_shared, "verify": _verify}[s["c"]["op"]](s)


# --- the definitions in 64 bits, written apart from the plain form -------------------------
def exact(c, seed):
    s = prepare(c, seed)
    return {"step_tables": _exact_tables, "attend_shared": _exact_attend, "verify": _exact_verify}[c["op"]](c, s)


def _exact_tables(c, s):
    kept, new, held = s["kept"].tolist(), s["new"].tolist(), s["held"].tolist()
    table, ring, (head, count) = s["table"].tolist(), s["ring"].tolist(), s["free"].tolist()
    prefix, size, asked, taken, given = s["prefix_table"].tolist(), s["pages"], 0, 0, 0
    starts, lens, positions, slots, left = [0], [], [], [], list(held)
    for i in range(c["n"]):
        length = kept[i] + new[i]
        need = math.ceil(length / PAGE)
        want = max(0, need - max(held[i], c["prefix"])) if need else 0
        asked += want
        fine = want == 0 or asked <= count
        if fine:
            for e in range(held[i], need):
                if e < c["prefix"]:
                    table[i][e] = prefix[e]
                else:
                    table[i][e] = ring[(head + taken) % size]
                    taken += 1
            for e in range(max(need, c["prefix"]), held[i]):
                ring[(head + count + given) % size] = table[i][e]
                given += 1
            left[i] = need
        lens.append(length if fine else 0)
        starts.append(starts[-1] + new[i])
        for at in range(kept[i], length):
            positions.append(at if fine else 0)
            slots.append(table[i][at // PAGE] * PAGE + at % PAGE if fine else -1)
    got = {"table": table, "ring": ring, "free_out": [(head + taken) % size, count - taken + given], "held_out": left,
           "row_start": starts, "seq_lens": lens, "positions": positions, "slots": slots}
    return {k: torch.tensor(v, dtype=s[k].dtype) for k, v in got.items()}


def _exact_verify(c, s):
    starts, tokens, u = s["row_start"].tolist(), s["tokens"].tolist(), s["u_accept"].double().tolist()
    out, accepted, kept = [-1] * s["n_rows"], [], []
    whole = lambda x: torch.floor(x.double() * 2.0 ** 40).long().cpu()  # noqa: E731
    for i in range(c["n"]):
        at, end = starts[i], starts[i + 1]
        while at < end - 1:
            token = tokens[at + 1]
            q = float(s["draft"][at, token]) if c["draft"] else 1.0
            if not u[at] * q < float(s["target"][at, token]):
                break
            out[at] = token
            at += 1
        w = target = whole(s["target"][at])
        if at < end - 1:
            if c["draft"]:
                w = target - whole(s["draft"][at])
            else:
                w = target.clone()
                w[tokens[at + 1]] = 0
            w = torch.where(w > 0, w, torch.zeros_like(w))
            if int(w.sum()) == 0:
                w = target
        threshold = int(float(s["u_sample"][i]) * 2.0 ** 32) * int(w.sum()) >> 32
        out[at] = int((w.cumsum(0) > threshold).nonzero()[0, 0])
        accepted.append(at - starts[i])
        kept.append(int(s["seq_lens"][i]) - (end - 1 - at))
    return {"out": torch.tensor(out, dtype=torch.int32), "accepted": torch.tensor(accepted, dtype=torch.int32),
            "kept": torch.tensor(kept, dtype=torch.int32)}


def _exact_attend(c, s):
    hkv, g, d, r, n = c["hkv"], c["hq"] // c["hkv"], c["d"], c["rows"], c["n"]
    out = torch.zeros((s["n_rows"], c["hq"], d), dtype=torch.float64, device="cuda")
    lens = s["seq_lens"].tolist()
    cached = lambda name, pages, h: (s[name + "_pool"][pages][:, :, h].double() * s[name + "_scale"][pages][:, h, None, None].double()).reshape(-1, d)  # noqa: E731
    for h in range(hkv):
        q = s["q"][:, h * g:(h + 1) * g].double() / math.sqrt(d)                  # [rows, g, d]
        pages = s["prefix_table"].long()
        x = torch.einsum("rgd,td->rgt", q, cached("k", pages, h))
        common = torch.logsumexp(x, -1)                                           # the shared tokens' share
        value = torch.softmax(x, -1).reshape(n * r * g, -1) @ cached("v", pages, h)
        value = value.view(n * r, g, d)
        del x
        for i in range(n):
            mine = s["table"][i, c["prefix"] // PAGE:_pages(lens[i])].long()
            held = lens[i] - c["prefix"]
            a, b = i * r, (i + 1) * r
            y = torch.einsum("rgd,td->rgt", q[a:b], cached("k", mine, h)[:held])
            later = torch.arange(held, device="cuda")[None] > torch.arange(held - r, held, device="cuda")[:, None]
            y = y.masked_fill(later[:, None], -math.inf)
            rest = torch.logsumexp(y, -1)
            both = torch.logaddexp(common[a:b], rest)
            own_value = torch.softmax(y, -1) @ cached("v", mine, h)[:held]
            out[a:b, h * g:(h + 1) * g] = (torch.exp(common[a:b] - both)[..., None] * value[a:b]
                                           + torch.exp(rest - both)[..., None] * own_value)
    return {"out": out}
