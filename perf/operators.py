"""Cases of the decode step's operators around the ternary projections: block
tables and slot maps from request lengths, the append of new keys and values to
a paged cache, attention of one new token per request over that cache, and the
penalties, biases and grammar masks on the output head's logits.

`run` computes a case in its plain form (elementary torch operations in 32
bits, rounded once at the end), or, where `own` is true, with the library.
Every size a case needs stands in the case; the seed gives the values and their
order (which request has which length, where pages lie in the pool).
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
E4M3_MAX = 448.0
VOCAB = 248320          # the output head's rows


# ------------------------------------------------------------------ cases ---
def _attention(name, requests, q_heads, kv_heads, head_dim, page, cache, shortest, longest, q="bf16", out="bf16",
               layout="tokens", empty=0, window=0):
    c = {"op": "attention", "requests": requests, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
         "page": page, "cache": cache, "shortest": shortest, "longest": longest, "q": q, "out": out, "layout": layout,
         "empty": empty, "window": window}
    return dict(c, name=name) if name else c


def _tables(name, requests, page, shortest, longest, new_shortest, new_longest, padding):
    c = {"op": "tables", "requests": requests, "page": page, "shortest": shortest, "longest": longest,
         "new_shortest": new_shortest, "new_longest": new_longest, "padding": padding}
    return dict(c, name=name) if name else c


def _append(name, tokens, kv_heads, head_dim, page, cache, src, layout="tokens"):
    c = {"op": "append", "tokens": tokens, "kv_heads": kv_heads, "head_dim": head_dim, "page": page, "cache": cache,
         "src": src, "layout": layout}
    return dict(c, name=name) if name else c


def _logits(name, rows, vocab, dtype, shortest, longest, biases):
    c = {"op": "logits", "rows": rows, "vocab": vocab, "dtype": dtype, "shortest": shortest, "longest": longest,
         "biases": biases}
    return dict(c, name=name) if name else c


def listed():
    return [
        # the first tokens of one conversation: nothing but latency (24 heads of 256 are the 6144-wide attention output)
        _attention("attention first tokens", 1, 24, 4, 256, 16, "bf16", 37, 37),
        # a chat server's ordinary batch, with two slots that hold no request
        _attention("attention chat batch", 32, 32, 8, 128, 16, "bf16", 200, 4500, empty=2),
        # one very long document: too few rows for the GPU unless its length is split
        _attention("attention one long", 1, 24, 4, 256, 64, "bf16", 131071, 131071),
        # a batch of long documents on an 8-bit cache
        _attention("attention long 8-bit", 16, 32, 8, 128, 32, "e4m3", 20000, 60000),
        # every head with keys of its own, an odd head width and page, a sliding window, an exact fp32 output
        _attention("attention own heads", 24, 16, 16, 80, 24, "f16", 1, 3001, q="f32", out="f32", layout="heads",
                   window=1999),
        # the largest: a full batch with eight query heads to a key head
        _attention("attention full batch", 128, 64, 8, 128, 16, "bf16", 1000, 16000),
        # the step's bookkeeping: one new token for each request of a captured batch
        _tables("tables decode", 64, 16, 100, 8000, 1, 1, 0),
        # admission of new prompts, some behind a cached prefix
        _tables("tables admission", 512, 16, 1, 4000, 1, 8192, 777),
        # the new keys and values of one decode step
        _append("append decode", 64, 8, 128, 16, "bf16", "bf16"),
        # a prompt's keys and values, straight from the fp32 projection
        _append("append prompt", 30011, 4, 256, 64, "bf16", "f32", layout="heads"),
        # one user's logits
        _logits("logits one", 1, VOCAB, "f32", 700, 700, 40),
        # a batch's logits
        _logits("logits batch", 64, VOCAB, "f32", 16, 8000, 300),
    ]


def _log(rng, low, high):
    """Evenly over the logarithm; never a multiple of 1024, which the listed cases' widths already are."""
    n = int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))
    return n + (n % 1024 == 0)


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "tables", "append", "logits"])
    if op == "attention":
        cache = rng.choice(["bf16", "bf16", "f16", "e4m3"])
        head_dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        kv_heads = rng.choice([1, 2, 4, 5, 8, 8, 16])
        group = rng.choice([1, 2, 3, 4, 6, 7, 8])
        page = rng.choice([8, 16, 16, 24, 32, 64, 128])
        requests = _log(rng, 1, 128)
        # at most 0.6e9 key elements even where every request has the longest length: under the largest listed case
        longest = max(2, min(_log(rng, 8, 200000), int(0.6e9 / (kv_heads * head_dim * requests))))
        shortest = min(longest, int(longest * rng.choice([0.01, 0.1, 0.5, 1.0])) | 1)
        q, out = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("f32", "f32"), ("f32", "bf16")])
        return _attention(None, requests, kv_heads * group, kv_heads, head_dim, page, cache, shortest, longest, q, out,
                          rng.choice(["tokens", "heads"]), rng.choice([0, 0, requests // 8]),
                          rng.choice([0, 0, longest // 3 | 1]))
    if op == "tables":
        requests = _log(rng, 1, 2000)
        new = rng.choice([1, 1, _log(rng, 1, 4000)])
        longest = _log(rng, 1, 20000)
        return _tables(None, requests, rng.choice([8, 16, 24, 32, 64, 128]), 1, longest, 1, new, rng.randrange(0, 300))
    if op == "append":
        return _append(None, _log(rng, 1, 30000), rng.choice([1, 2, 4, 5, 8, 16]), rng.choice([64, 80, 96, 128, 256]),
                       rng.choice([8, 16, 24, 64]), rng.choice(["bf16", "f16", "e4m3"]), rng.choice(["f32", "bf16", "f16"]),
                       rng.choice(["tokens", "heads"]))
    longest = _log(rng, 1, 16000)
    return _logits(None, _log(rng, 1, 64), rng.choice([VOCAB, _log(rng, 1000, VOCAB)]), rng.choice(["f32", "f32", "bf16"]),
                   min(longest, int(longest * rng.choice([0.01, 0.5, 1.0])) | 1), longest, _log(rng, 1, 500))


# ----------------------------------------------------------------- inputs ---
def _spread(shortest, longest, count):
    """`count` lengths from shortest to longest, evenly over their logarithm."""
    if count == 1:
        return [longest]
    return [int(round(shortest * (longest / shortest) ** (i / (count - 1)))) for i in range(count)]


def _lengths(case):
    n = _spread(case["shortest"], case["longest"], case["requests"])
    return [0] * case["empty"] + n[case["empty"]:]


def _news(case):
    return _spread(case["new_shortest"], case["new_longest"], case["requests"])


def _pages(n, page):
    return -(-n // page)


def _pool(pages, page, kv_heads, head_dim, layout, fill):
    """A cache tensor, indexed [page][token][head][element] whatever its order in memory."""
    if layout == "heads":
        return fill((pages, kv_heads, page, head_dim)).permute(0, 2, 1, 3)
    return fill((pages, page, kv_heads, head_dim))


def _handle(state, case, requests=0, q_heads=0):
    import bit_gemv_gb300 as nt
    state["cache"] = nt.KvCache(state["k"], state["v"], state["k_scale"], state["v_scale"])
    if requests:
        state["workspace"] = torch.empty(nt.ninfer_kv_attention_workspace(state["cache"], requests, q_heads),
                                         dtype=torch.uint8, device="cuda")


def _stored(case, gen, spread):
    """A filler of cache values; an 8-bit cache stores them divided by its scale."""
    dtype = DTYPES[case["cache"]]

    def fill(shape):
        if case["cache"] == "e4m3":
            return (torch.randn(shape, generator=gen, device="cuda", dtype=torch.bfloat16) * spread).to(dtype)
        return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)
    return fill


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    return {"attention": _prepare_attention, "tables": _prepare_tables, "append": _prepare_append,
            "logits": _prepare_logits}[case["op"]](case, gen, rng)


def _prepare_attention(case, gen, rng):
    lengths = rng.permutation(np.array(_lengths(case), np.int64))
    page, used = case["page"], -(-lengths // case["page"])
    width, total = max(1, int(used.max())), int(used.sum())
    pool = rng.permutation(total + 7)
    table = np.full((len(lengths), width), -1, np.int64)
    table[np.arange(width)[None, :] < used[:, None]] = pool[:total]
    scaled = case["cache"] == "e4m3"
    state = {"op": case["op"], "page": page, "window": case["window"], "scale": case["head_dim"] ** -0.5,
             "k_scale": 0.0625 if scaled else 1.0, "v_scale": 0.03125 if scaled else 1.0, "out_dtype": DTYPES[case["out"]],
             "longest": max(lengths), "lengths": torch.from_numpy(lengths.astype(np.int32)).cuda(),
             "table": torch.from_numpy(table.astype(np.int32)).cuda()}
    args = (total + 7, page, case["kv_heads"], case["head_dim"], case["layout"])
    state["k"] = _pool(*args, _stored(case, gen, 16.0))
    state["v"] = _pool(*args, _stored(case, gen, 32.0))
    # queries somewhat larger than keys, so that some scores stand out as trained heads' do
    q = torch.randn((len(lengths), case["q_heads"], case["head_dim"]), generator=gen, device="cuda") * 1.5
    state["q"] = q.to(DTYPES[case["q"]])
    shape = (len(lengths), case["q_heads"])
    state["out"] = torch.empty(shape + (case["head_dim"],), dtype=state["out_dtype"], device="cuda")
    state["lse"] = torch.empty(shape, dtype=torch.float32, device="cuda")
    if own:
        _handle(state, case, len(lengths), case["q_heads"])
    return state


def _prepare_tables(case, gen, rng):
    page = case["page"]
    lengths = rng.permutation(np.array(_spread(case["shortest"], case["longest"], case["requests"]), np.int64))
    new = rng.permutation(np.array(_news(case), np.int64))
    held, last = -(-lengths // page), -(-(lengths + new) // page)
    pool = rng.permutation(int(last.sum()) + 11)
    table = np.full((len(lengths), _pages(case["longest"] + case["new_longest"], page) + 3), -1, np.int64)
    table[np.arange(table.shape[1])[None, :] < held[:, None]] = pool[:int(held.sum())]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    state = {"op": case["op"], "page": page, "capacity": int(new.sum()) + case["padding"], "lengths": i32(lengths),
             "new": i32(new), "table": i32(table), "free": i32(pool[int(held.sum()):]), "buffers": None}
    if own:
        import bit_gemv_gb300 as nt
        state["buffers"] = nt.KvTables.empty(state["table"], state["capacity"])
    return state


def _prepare_append(case, gen, rng):
    tokens, page = case["tokens"], case["page"]
    pages = 2 * _pages(tokens, page) + 3
    scaled = case["cache"] == "e4m3"
    state = {"op": case["op"], "page": page, "k_scale": 0.0625 if scaled else 1.0, "v_scale": 0.03125 if scaled else 1.0}
    args = (pages, page, case["kv_heads"], case["head_dim"], case["layout"])
    state["k"], state["v"] = _pool(*args, _stored(case, gen, 16.0)), _pool(*args, _stored(case, gen, 32.0))
    # keys and values are slices of one projection's rows, which hold the queries too; the tokens' slots run through pages
    width = case["kv_heads"] * case["head_dim"]
    rows = torch.randn((tokens, 4 * width), generator=gen, device="cuda").to(DTYPES[case["src"]])
    state["k_new"] = rows[:, 2 * width:3 * width].unflatten(1, (case["kv_heads"], case["head_dim"]))
    state["v_new"] = rows[:, 3 * width:].unflatten(1, (case["kv_heads"], case["head_dim"]))
    runs = rng.permutation(pages)[:_pages(tokens, page) + 1]
    slots = (runs[:, None] * page + np.arange(page)[None, :]).reshape(-1)
    state["slots"] = torch.from_numpy(slots[page // 2:page // 2 + tokens].astype(np.int64)).cuda()
    if own:
        _handle(state, case)
    return state


def _prepare_logits(case, gen, rng):
    rows, vocab = case["rows"], case["vocab"]
    lengths = rng.permutation(np.array(_spread(case["shortest"], case["longest"], rows), np.int64))
    f = lambda a: torch.from_numpy(np.asarray(a, np.float32)).cuda()  # noqa: E731
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    u = torch.rand((rows, case["longest"]), generator=gen, device="cuda")
    history = (vocab * u ** 3).to(torch.int32).clamp_(max=vocab - 1)      # a few tokens come again and again
    each = min(case["biases"], vocab)
    ids = np.concatenate([rng.choice(vocab, each, replace=False) for _ in range(rows)])
    words = _pages(vocab, 32)
    mask = torch.randint(-2 ** 31, 2 ** 31, (3, words), generator=gen, device="cuda").to(torch.int32)
    mask[2] &= mask[1] << 1
    state = {"op": case["op"], "lengths": i32(lengths), "history": history, "prompts": i32(lengths // 3),
             "logits": (torch.randn((rows, vocab), generator=gen, device="cuda") * 3).to(DTYPES[case["dtype"]]),
             "repetition": f(rng.uniform(1.0, 1.3, rows)), "presence": f(rng.uniform(0, 0.8, rows)),
             "frequency": f(rng.uniform(-0.1, 0.5, rows)), "bias_ids": i32(ids),
             "bias_offsets": i32(np.arange(rows + 1) * each), "bias_values": f(rng.normal(0, 4, ids.size)),
             "mask": mask, "mask_rows": i32(rng.integers(-1, 3, rows))}
    state["out"] = torch.empty_like(state["logits"])
    return state


# -------------------------------------------------------------------- run ---
def run(state):
    return {"attention": _run_attention, "tables": _run_tables, "append": _run_append,
            "logits": _run_logits}[state["op"]](state)


def _rows_of(pool, page, token):
    """pool[page][token] for any element type."""
    if pool.element_size() == 1:
        return pool.view(torch.uint8)[page, token].view(pool.dtype)
    return pool[page, token]


def _run_attention(s):
    if own:
        import bit_gemv_gb300 as nt
        nt.ninfer_kv_attention(s["q"], s["cache"], s["table"], s["lengths"], scale=s["scale"], window=s["window"],
                               out=s["out"], lse=s["lse"], workspace=s["workspace"])
        return {"out": s["out"], "lse": s["lse"]}
    key = torch.arange(int(s["longest"]), device="cuda")
    page, token = s["table"].long()[:, key // s["page"]].clamp_(min=0), (key % s["page"])[None, :]
    kv_heads, head_dim = s["k"].shape[2:]
    q = s["q"].float().unflatten(1, (kv_heads, -1))
    k = _rows_of(s["k"], page, token).float()
    score = torch.einsum("rhgd,rlhd->rhgl", q, k) * (s["scale"] * s["k_scale"])
    del k
    length = s["lengths"][:, None]
    seen = key[None, :] < length
    if s["window"]:
        seen &= key[None, :] >= length - s["window"]
    score = score.masked_fill(~seen[:, None, None, :], -math.inf)
    top = score.amax(-1, keepdim=True)
    weight = torch.exp(score - torch.where(top == -math.inf, 0.0, top))
    total = weight.sum(-1, keepdim=True)
    v = _rows_of(s["v"], page, token).float()
    out = torch.einsum("rhgl,rlhd->rhgd", weight, v) * s["v_scale"] / torch.where(total > 0, total, 1.0)
    lse = (top + torch.log(total)).squeeze(-1)
    return {"out": out.flatten(1, 2).to(s["out_dtype"]), "lse": lse.flatten(1, 2)}


def _run_tables(s):
    if own:
        import bit_gemv_gb300 as nt
        t = nt.ninfer_kv_tables(s["lengths"], s["new"], s["page"], s["free"], s["table"], s["capacity"], out=s["buffers"])
        return {"table": t.block_table, "slots": t.slots, "positions": t.positions, "rows": t.token_rows,
                "offsets": t.offsets, "lengths": t.lengths, "counts": t.counts}
    page, old, new, table, free = s["page"], s["lengths"].long(), s["new"].long(), s["table"], s["free"]
    held, last = (old + page - 1) // page, (old + new + page - 1) // page
    zero = torch.zeros(1, dtype=torch.long, device="cuda")
    offsets = torch.cat([zero, torch.cumsum(new, 0)])
    taken = torch.cat([zero, torch.cumsum(last - held, 0)])
    column = torch.arange(table.shape[1], device="cuda")[None, :]
    fresh = (column >= held[:, None]) & (column < last[:, None])
    at = (taken[:-1, None] + column - held[:, None]).clamp_(0, len(free) - 1)
    table = torch.where(fresh, free[at], table)
    token = torch.arange(s["capacity"], device="cuda")
    real = token < offsets[-1]
    row = torch.searchsorted(offsets[1:], token, right=True).clamp_(max=len(old) - 1)
    position = old[row] + token - offsets[row]
    slots = table[row, (position // page).clamp_(max=table.shape[1] - 1)].long() * page + position % page
    pad = lambda x: torch.where(real, x, -1)  # noqa: E731
    return {"table": table, "slots": pad(slots), "positions": pad(position).int(), "rows": pad(row).int(),
            "offsets": offsets.int(), "lengths": (old + new).int(), "counts": torch.stack([offsets[-1], taken[-1]]).int()}


def _run_append(s):
    if own:
        import bit_gemv_gb300 as nt
        nt.ninfer_kv_append(s["cache"], s["k_new"], s["v_new"], s["slots"])
        return {"k": s["k"], "v": s["v"]}
    page, token = s["slots"] // s["page"], s["slots"] % s["page"]
    _put(s["k"], page, token, s["k_new"].float() / s["k_scale"])
    _put(s["v"], page, token, s["v_new"].float() / s["v_scale"])
    return {"k": s["k"], "v": s["v"]}


def _put(pool, page, token, x):
    if pool.element_size() == 1:
        pool.view(torch.uint8)[page, token] = x.clamp(-E4M3_MAX, E4M3_MAX).to(pool.dtype).view(torch.uint8)
    else:
        pool[page, token] = x.to(pool.dtype)


def _run_logits(s):
    if own:
        import bit_gemv_gb300 as nt
        return nt.ninfer_logits_process(
            s["logits"], out=s["out"], history=s["history"], history_lengths=s["lengths"], prompt_lengths=s["prompts"],
            repetition=s["repetition"], presence=s["presence"], frequency=s["frequency"], bias_offsets=s["bias_offsets"],
            bias_ids=s["bias_ids"], bias_values=s["bias_values"], mask=s["mask"], mask_rows=s["mask_rows"])
    x = s["logits"].float()
    place = torch.arange(s["history"].shape[1], device="cuda")[None, :]
    seen = place < s["lengths"][:, None]
    told = seen & (place >= s["prompts"][:, None])
    ids = s["history"].long()
    both = torch.zeros((2,) + x.shape, device="cuda")
    both[0].scatter_add_(1, ids, seen.float())
    both[1].scatter_add_(1, ids, told.float())
    column = lambda name: s[name][:, None]  # noqa: E731
    scaled = torch.where(x > 0, x / column("repetition"), x * column("repetition"))
    x = torch.where(both[0] > 0, scaled, x)
    x = x - column("frequency") * both[1] - column("presence") * (both[1] > 0)
    entry = torch.arange(len(s["bias_ids"]), device="cuda")
    row = torch.searchsorted(s["bias_offsets"][1:].long(), entry, right=True)
    x = x.index_put((row, s["bias_ids"].long()), s["bias_values"], accumulate=True)
    token = torch.arange(x.shape[1], device="cuda")
    bit = (s["mask"][:, token // 32] >> (token % 32)) & 1
    allowed = (bit[s["mask_rows"].long().clamp(min=0)] != 0) | (s["mask_rows"][:, None] < 0)
    return torch.where(allowed, x, -math.inf).to(s["logits"].dtype)


# ------------------------------------------------------------------- work ---
def work(case):
    if case["op"] == "attention":
        lengths = _lengths(case)
        keys = sum(min(n, case["window"]) if case["window"] else n for n in lengths)
        rows = case["requests"] * case["q_heads"]
        table = sum(_pages(min(n, case["window"]) if case["window"] else n, case["page"]) for n in lengths)
        return {"bytes": 2 * keys * case["kv_heads"] * case["head_dim"] * BYTES[case["cache"]] + 4 * table
                + 4 * case["requests"] + rows * (case["head_dim"] * (BYTES[case["q"]] + BYTES[case["out"]]) + 4),
                "flops": 4 * keys * case["q_heads"] * case["head_dim"]}
    if case["op"] == "tables":
        tokens = sum(_news(case))
        pages = tokens // case["page"]
        return {"bytes": 16 * (tokens + case["padding"]) + 8 * pages + 16 * case["requests"], "flops": 0}
    if case["op"] == "append":
        width = case["kv_heads"] * case["head_dim"]
        return {"bytes": case["tokens"] * (2 * width * (BYTES[case["src"]] + BYTES[case["cache"]]) + 8), "flops": 0}
    rows, vocab = case["rows"], case["vocab"]
    history = sum(_spread(case["shortest"], case["longest"], rows))
    return {"bytes": rows * vocab * 2 * BYTES[case["dtype"]] + 3 * vocab // 8 + 4 * history + 8 * rows * case["biases"],
            "flops": 0}


# ------------------------------------------------------------------ exact ---
def exact(case, seed):
    """The definitions in 64 bits, request by request; whole numbers have no such value."""
    if case["op"] == "tables":
        return None
    s = prepare(case, seed)
    if case["op"] == "append":
        return {"k": _exact_append(s, "k"), "v": _exact_append(s, "v")}
    if case["op"] == "logits":
        return torch.stack([_exact_logits_row(s, b) for b in range(case["rows"])])
    rows = [_exact_attention_row(s, r, int(n)) for r, n in enumerate(s["lengths"].tolist())]
    return {"out": torch.stack([r[0] for r in rows]), "lse": torch.stack([r[1] for r in rows])}


def _wide(x):
    return x.float().double()


def _exact_attention_row(s, r, length):
    q = _wide(s["q"][r])
    first = max(0, length - s["window"]) if s["window"] else 0
    if length == 0:
        return torch.zeros_like(q), torch.full((q.shape[0],), -math.inf, dtype=torch.float64, device="cuda")
    pages = s["table"][r, :_pages(length, s["page"])].long()

    def held(pool, scale):
        rows = (pool.view(torch.uint8) if pool.element_size() == 1 else pool)[pages].flatten(0, 1)[first:length]
        return _wide(rows.view(pool.dtype)) * scale
    k, v = held(s["k"], s["k_scale"]), held(s["v"], s["v_scale"])
    group = q.shape[0] // k.shape[1]
    out, lse = torch.empty_like(q), torch.empty(q.shape[0], dtype=torch.float64, device="cuda")
    for h in range(k.shape[1]):
        heads = slice(h * group, (h + 1) * group)
        score = q[heads] @ k[:, h].T * s["scale"]
        lse[heads] = torch.logsumexp(score, 1)
        out[heads] = torch.exp(score - lse[heads][:, None]) @ v[:, h]
    return out, lse


def _exact_append(s, which):
    pool = _wide(s[which])
    flat = s["slots"]
    pool[flat // s["page"], flat % s["page"]] = _wide(s[which + "_new"]) / s[which + "_scale"]
    return pool


def _exact_logits_row(s, b):
    x = _wide(s["logits"][b])
    history = s["history"][b, :int(s["lengths"][b])].long()
    r, p, f = (float(s[n][b]) for n in ("repetition", "presence", "frequency"))
    ids = torch.unique(history)
    x[ids] = torch.where(x[ids] > 0, x[ids] / r, x[ids] * r)
    ids, times = torch.unique(history[int(s["prompts"][b]):], return_counts=True)
    x[ids] -= f * times + p
    part = slice(int(s["bias_offsets"][b]), int(s["bias_offsets"][b + 1]))
    x[s["bias_ids"][part].long()] += s["bias_values"][part].double()
    row = int(s["mask_rows"][b])
    if row >= 0:
        bits = np.unpackbits(s["mask"][row].cpu().numpy().view(np.uint8), bitorder="little")[:x.numel()]
        x[torch.from_numpy(bits == 0).cuda()] = -math.inf
    return x
