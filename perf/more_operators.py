"""Cases of the operators that complete a model's step around the projections, the
cache and the logit controls: root-mean-square norm with the residual's addition,
rotary positions of queries and keys, the gated delta rule over a state per head
(one token a request, and whole prompts), and the choice of the next token.

`run` computes a case in its plain form (elementary torch operations in 32 bits,
in 64 for angles and for the running sums of the choice, rounded once at the end),
or, where `own` is true, with the library. Every size a case needs stands in the
case; the seed gives the values and their order.
"""
import math

import numpy as np
import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
BYTES = {"f32": 4, "bf16": 2, "f16": 2}
VOCAB = 248320          # the output head's rows
HIDDEN = 5120
EPS = 1e-6
CHUNK = 64              # tokens that the plain form of the gated delta rule takes at once


# ------------------------------------------------------------------ cases ---
def _norm(name, rows, cols, x, residual, out, group=0, gate=False, weight="bf16"):
    c = {"op": "norm", "rows": rows, "cols": cols, "x": x, "residual": residual, "out": out, "group": group or cols,
         "gate": gate, "weight": weight}
    return dict(c, name=name) if name else c


def _rotary(name, tokens, q_heads, kv_heads, head_dim, rotary_dim, dtype, interleaved, normed, factor, longest):
    c = {"op": "rotary", "tokens": tokens, "q_heads": q_heads, "kv_heads": kv_heads, "head_dim": head_dim,
         "rotary_dim": rotary_dim, "dtype": dtype, "interleaved": interleaved, "normed": normed, "factor": factor,
         "longest": longest}
    return dict(c, name=name) if name else c


def _delta(name, requests, shortest, longest, k_heads, v_heads, k_dim, v_dim, dtype="bf16", out="bf16", fresh=0):
    c = {"op": "delta", "requests": requests, "shortest": shortest, "longest": longest, "k_heads": k_heads,
         "v_heads": v_heads, "k_dim": k_dim, "v_dim": v_dim, "dtype": dtype, "out": out, "fresh": fresh}
    return dict(c, name=name) if name else c


def _sample(name, rows, vocab, dtype, controls):
    c = {"op": "sample", "rows": rows, "vocab": vocab, "dtype": dtype, "controls": controls}
    return dict(c, name=name) if name else c


def listed():
    return [
        # one user's token between two projections: nothing but latency
        _norm("norm token", 1, HIDDEN, "f32", "f32", "bf16"),
        # a prompt's rows on a 16-bit residual stream
        _norm("norm prompt", 8192, HIDDEN, "bf16", "bf16", "bf16"),
        # the gated norm behind the delta rule: 48 heads of 128 with one weight, gates from a projection's rows
        _norm("norm gated heads", 4001, 6144, "bf16", "", "bf16", group=128, gate=True, weight="f32"),
        # one step of a batch: 24 / 4 heads of 256, a quarter of each rotated, queries and keys normed
        _rotary("rotary step", 64, 24, 4, 256, 64, "bf16", False, True, 1.0, 100000),
        # a prompt of a scaled long context, whole heads, neighbouring pairs
        _rotary("rotary prompt", 30011, 32, 8, 128, 128, "bf16", True, False, 8.0, 1000000),
        # one user's token: 16 key heads and 48 value heads of 128
        _delta("delta token", 1, 1, 1, 16, 48, 128, 128),
        # a full batch of single tokens: the states' bytes
        _delta("delta batch", 64, 1, 1, 16, 48, 128, 128),
        # prompts of very different lengths beside single tokens, some of them new; small uneven heads, exact types
        _delta("delta ragged", 24, 1, 1201, 6, 12, 96, 64, "f32", "f32", fresh=7),
        # one long prompt
        _delta("delta prompt", 1, 8001, 8001, 16, 48, 128, 128, fresh=1),
        # one user's next token
        _sample("sample one", 1, VOCAB, "f32", "top_p"),
        # a batch whose users chose differently: greedy, temperature alone, top-k, top-p, min-p
        _sample("sample batch", 64, VOCAB, "f32", "mixed"),
        # many users of a small vocabulary, 16-bit logits with their many ties
        _sample("sample small vocabulary", 256, 32003, "bf16", "top_k"),
    ]


def _log(rng, low, high):
    """Evenly over the logarithm."""
    return int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))


def draw(rng):
    op = rng.choice(["norm", "rotary", "delta", "delta", "sample", "sample"])
    if op == "norm":
        group = rng.choice([0, 0, 64, 96, 128])
        step = rng.choice([1, 8, 8])
        cols = group * rng.randrange(1, 49) if group else _log(rng, 64, 16384) // step * step
        rows = min(_log(rng, 1, 20000), max(1, 40000000 // cols))
        return _norm(None, rows, cols, rng.choice(["f32", "bf16", "f16"]), rng.choice(["", "f32", "bf16"]),
                     rng.choice(["f32", "bf16", "bf16", "f16"]), group, group > 0 and rng.random() < 0.5,
                     rng.choice(["f32", "bf16"]))
    if op == "rotary":
        head_dim = rng.choice([64, 80, 96, 128, 128, 192, 256])
        rotary_dim = rng.choice([head_dim, head_dim, head_dim // 2, head_dim // 4])
        kv_heads = rng.choice([1, 2, 4, 8])
        q_heads = kv_heads * rng.choice([1, 2, 3, 4, 6, 8])
        tokens = min(_log(rng, 1, 30000), 150000000 // ((q_heads + kv_heads) * head_dim))
        return _rotary(None, tokens, q_heads, kv_heads, head_dim, rotary_dim, rng.choice(["bf16", "bf16", "f16", "f32"]),
                       rng.random() < 0.5, rng.random() < 0.5, rng.choice([1.0, 4.0, 32.0]), _log(rng, 100, 2000000))
    if op == "delta":
        k_heads = rng.choice([1, 2, 4, 8, 16])
        v_heads = k_heads * rng.choice([1, 2, 3, 4])
        k_dim, v_dim = rng.choice([(64, 64), (128, 128), (128, 128), (96, 160), (128, 256), (256, 128), (48, 80)])
        requests = _log(rng, 1, 64)
        # at most as many head tokens as the longest listed prompt, and no more state than the listed batch
        longest = rng.choice([1, 1, _log(rng, 1, 6000)])
        longest = max(1, min(longest, 300000 // (requests * v_heads)))
        requests = min(requests, max(1, 3000 * 16384 // (v_heads * k_dim * v_dim)))
        dtype, out = rng.choice([("bf16", "bf16"), ("bf16", "f32"), ("f16", "f16"), ("f32", "f32")])
        return _delta(None, requests, max(1, longest // rng.choice([1, 2, 50])), longest, k_heads, v_heads, k_dim, v_dim,
                      dtype, out, rng.choice([0, requests // 2]))
    return _sample(None, _log(rng, 1, 64), rng.choice([VOCAB, _log(rng, 100, VOCAB)]), rng.choice(["f32", "f32", "bf16", "f16"]),
                   rng.choice(["mixed", "plain", "top_p", "top_k", "min_p"]))


# ----------------------------------------------------------------- inputs ---
def _spread(shortest, longest, count):
    """`count` lengths from shortest to longest, evenly over their logarithm."""
    if count == 1:
        return [longest]
    return [int(round(shortest * (longest / shortest) ** (i / (count - 1)))) for i in range(count)]


def _news(case):
    return _spread(case["shortest"], case["longest"], case["requests"])


def prepare(case, seed):
    gen = torch.Generator("cuda")
    gen.manual_seed(seed)
    rng = np.random.default_rng(seed)
    return {"norm": _prepare_norm, "rotary": _prepare_rotary, "delta": _prepare_delta,
            "sample": _prepare_sample}[case["op"]](case, gen, rng)


def _randn(gen, *shape):
    return torch.randn(shape, generator=gen, device="cuda")


def _prepare_norm(case, gen, rng):
    rows, cols = case["rows"], case["cols"]
    s = {"op": "norm", "group": case["group"], "residual": None, "sum": None, "gate": None,
         "x": _randn(gen, rows, cols).to(DTYPES[case["x"]]),
         "weight": (1 + 0.2 * _randn(gen, case["group"])).to(DTYPES[case["weight"]]),
         "out": torch.empty((rows, cols), dtype=DTYPES[case["out"]], device="cuda")}
    if case["residual"]:
        # a residual stream is larger than what one layer adds to it
        s["residual"] = (_randn(gen, rows, cols) * 4).to(DTYPES[case["residual"]])
        s["sum"] = torch.empty_like(s["residual"])
    if case["gate"]:
        # the second half of a projection's rows
        s["gate"] = _randn(gen, rows, 2 * cols).to(DTYPES[case["x"]])[:, cols:]
    return s


def _frequencies(rotary_dim, factor):
    """Radians a position and the magnitude, in 64 bits: scaled by parts, the slow pairs by the factor, the fast ones not."""
    base, context, fast, slow = 1e6, 32768, 32.0, 1.0
    i = np.arange(rotary_dim // 2, dtype=np.float64)
    f = base ** (-2 * i / rotary_dim)
    if factor == 1.0:
        return f, 1.0
    at = [rotary_dim * math.log(context / (r * 2 * math.pi)) / (2 * math.log(base)) for r in (fast, slow)]
    first, last = max(math.floor(at[0]), 0), min(math.ceil(at[1]), rotary_dim - 1)
    ramp = np.clip((i - first) / max(last - first, 0.001), 0, 1)
    return f / factor * ramp + f * (1 - ramp), 0.1 * math.log(factor) + 1


def _prepare_rotary(case, gen, rng):
    tokens, q_heads, kv_heads, dim = case["tokens"], case["q_heads"], case["kv_heads"], case["head_dim"]
    rows = _randn(gen, tokens, q_heads + 2 * kv_heads, dim).to(DTYPES[case["dtype"]])     # one projection's rows
    first = rng.integers(0, max(1, case["longest"] - tokens), 1)[0]
    positions = first + np.arange(tokens) if tokens > 64 else rng.integers(0, case["longest"], tokens)
    f, magnitude = _frequencies(case["rotary_dim"], case["factor"])
    s = {"op": "rotary", "rotary_dim": case["rotary_dim"], "interleaved": case["interleaved"], "q": rows[:, :q_heads],
         "k": rows[:, q_heads:q_heads + kv_heads], "positions": torch.from_numpy(positions.astype(np.int32)).cuda(),
         "radians": torch.from_numpy(f).cuda(), "magnitude": float(np.float32(magnitude)), "q_weight": None, "k_weight": None}
    s["q_out"], s["k_out"] = (torch.empty(s[n].shape, dtype=rows.dtype, device="cuda") for n in "qk")
    if case["normed"]:
        s["q_weight"], s["k_weight"] = (1 + 0.2 * _randn(gen, 2, dim)).to(DTYPES[case["dtype"]])
    if own:
        import bit_gemv_gb300 as nt
        table, magnitude = nt.ninfer_rotary_frequencies(
            case["rotary_dim"], 1e6, "none" if case["factor"] == 1.0 else "dimensions", factor=case["factor"], context=32768)
        s["frequencies"], s["magnitude"] = torch.from_numpy(table).cuda(), magnitude
    return s


def _prepare_delta(case, gen, rng):
    news = rng.permutation(np.array(_news(case), np.int64))
    tokens, requests = int(news.sum()), case["requests"]
    k_heads, v_heads, k_dim, v_dim = case["k_heads"], case["v_heads"], case["k_dim"], case["v_dim"]
    i32 = lambda a: torch.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    width = 2 * k_heads * k_dim
    rows = _randn(gen, tokens, width + v_heads * v_dim).to(DTYPES[case["dtype"]])          # one projection's rows
    heads = lambda a, n: a.unflatten(1, (n, -1))  # noqa: E731
    held = rng.integers(1, 5000, requests)
    held[rng.permutation(requests)[:case["fresh"]]] = 0
    s = {"op": "delta", "q": heads(rows[:, :width // 2], k_heads), "k": heads(rows[:, width // 2:width], k_heads),
         "v": heads(rows[:, width:], v_heads), "scale": k_dim ** -0.5, "eps": EPS, "longest": int(news.max()),
         "single": case["longest"] == 1, "lengths": i32(held),
         # heads remember from a few tokens to thousands
         "log_decay": -torch.exp(_randn(gen, tokens, v_heads) - 3 - 3 * torch.rand(v_heads, generator=gen, device="cuda")),
         "beta": torch.sigmoid(_randn(gen, tokens, v_heads)),
         "slots": i32(rng.permutation(requests + 3)[:requests]), "offsets": i32(np.concatenate([[0], np.cumsum(news)])),
         "state": _randn(gen, requests + 3, v_heads, k_dim, v_dim) * 0.3,
         "out": torch.empty((tokens, v_heads, v_dim), dtype=DTYPES[case["out"]], device="cuda"), "workspace": None}
    if own:
        import bit_gemv_gb300 as nt
        need = nt.ninfer_gated_delta_workspace(tokens, requests, k_heads, v_heads, k_dim, v_dim)
        s["workspace"] = torch.empty(max(need, 1), dtype=torch.uint8, device="cuda")
    return s


KINDS = ("greedy", "plain", "top_p", "top_k", "min_p")


def _prepare_sample(case, gen, rng):
    rows, vocab = case["rows"], case["vocab"]
    x = _randn(gen, rows, vocab) * 2.2
    # beside the bulk a few tokens that fit, from far above all others to not quite
    fit = torch.rand((rows, vocab), generator=gen, device="cuda") * max(1.0, vocab / 64)
    x += torch.where(fit < 1, 16 * fit ** 3, 0.0)
    kinds = [KINDS[i % 5] for i in range(rows)] if case["controls"] == "mixed" else [case["controls"]] * rows
    kinds = [kinds[i] for i in rng.permutation(rows)]
    f = lambda low, high, *on: torch.from_numpy(np.where(np.isin(kinds, on), rng.uniform(low, high, rows), 0).astype(np.float32)).cuda()  # noqa: E731
    top_p = f(0.8, 0.98, "top_p", "top_k")
    return {"op": "sample", "logits": x.to(DTYPES[case["dtype"]]), "temperature": f(0.5, 1.2, *KINDS[1:]),
            "top_k": torch.from_numpy(np.where(np.isin(kinds, ["top_k"]), rng.integers(10, 200, rows), 0).astype(np.int32)).cuda(),
            "top_p": torch.where(top_p > 0, top_p, 1.0), "min_p": f(0.02, 0.1, "min_p"),
            "random": torch.rand(rows, generator=gen, device="cuda"),
            "tokens": torch.empty(rows, dtype=torch.int32, device="cuda"), "logprobs": torch.empty(rows, device="cuda")}


# -------------------------------------------------------------------- run ---
def run(state):
    return {"norm": _run_norm, "rotary": _run_rotary, "delta": _run_delta, "sample": _run_sample}[state["op"]](state)


def _run_norm(s):
    if own:
        import bit_gemv_gb300 as nt
        nt.ninfer_norm(s["x"], s["weight"], EPS, residual=s["residual"], sum=s["sum"], gate=s["gate"], group=s["group"],
                       out=s["out"])
        return {"out": s["out"], "sum": s["sum"]}
    x = s["x"].float()
    total = None
    if s["residual"] is not None:
        x = x + s["residual"].float()
        total = x.to(s["residual"].dtype)
    heads = x.unflatten(1, (-1, s["group"]))
    y = heads * torch.rsqrt(heads.square().mean(-1, keepdim=True) + EPS) * s["weight"].float()
    y = y.flatten(1)
    if s["gate"] is not None:
        z = s["gate"].float()
        y = y * (z / (1 + torch.exp(-z)))
    return {"out": y.to(s["out"].dtype), "sum": total}


def _rotated(s, x, weight):
    n, half = s["rotary_dim"], s["rotary_dim"] // 2
    y = x.float()
    if weight is not None:
        y = y * torch.rsqrt(y.square().mean(-1, keepdim=True) + EPS) * weight.float()
    angle = (s["positions"].double()[:, None] * s["radians"]).remainder(2 * math.pi)
    c, d = (t.float()[:, None] * s["magnitude"] for t in (torch.cos(angle), torch.sin(angle)))
    a, b = (y[..., 0:n:2], y[..., 1:n:2]) if s["interleaved"] else (y[..., :half], y[..., half:n])
    pair = a * c - b * d, b * c + a * d
    turned = torch.stack(pair, -1).flatten(-2) if s["interleaved"] else torch.cat(pair, -1)
    return torch.cat([turned, y[..., n:]], -1).to(x.dtype)


def _run_rotary(s):
    if own:
        import bit_gemv_gb300 as nt
        nt.ninfer_rotary(s["q"], s["k"], s["positions"], s["frequencies"], s["magnitude"], interleaved=s["interleaved"],
                         q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS, q_out=s["q_out"], k_out=s["k_out"])
        return {"q": s["q_out"], "k": s["k_out"]}
    return {"q": _rotated(s, s["q"], s["q_weight"]), "k": _rotated(s, s["k"], s["k_weight"])}


def _run_delta(s):
    if own:
        import bit_gemv_gb300 as nt
        nt.ninfer_gated_delta(s["q"], s["k"], s["v"], s["log_decay"], s["beta"], s["state"],
                              offsets=None if s["single"] else s["offsets"], slots=s["slots"], lengths=s["lengths"],
                              scale=s["scale"], norm_eps=s["eps"], out=s["out"], workspace=s["workspace"])
        return {"out": s["out"], "state": s["state"]}
    # tokens as (request, head, place), padded to whole chunks with tokens that change nothing
    size = min(CHUNK, s["longest"])
    longest = -(-s["longest"] // size) * size
    place = torch.arange(longest, device="cuda")[None, :]
    begin, count = s["offsets"][:-1].long()[:, None], s["offsets"].diff().long()[:, None]
    real = place < count
    at = (begin + place).clamp_(max=len(s["v"]) - 1)
    group = s["v"].shape[1] // s["k"].shape[1]
    rows = lambda x: (x.float()[at] * real[..., None, None]).transpose(1, 2)  # noqa: E731
    unit = lambda x: x * torch.rsqrt(x.square().sum(-1, keepdim=True) + s["eps"])  # noqa: E731
    q, k = (unit(rows(s[n])).repeat_interleave(group, 1) for n in "qk")
    v = rows(s["v"])
    beta, decay = ((s[n][at] * real[..., None]).transpose(1, 2) for n in ("beta", "log_decay"))
    state = s["state"][s["slots"].long()] * (s["lengths"] > 0)[:, None, None, None]
    lower = torch.ones(size, size, dtype=torch.bool, device="cuda").tril()
    eye = torch.eye(size, device="cuda")
    outs = []
    for i in range(0, longest, size):       # the state goes from chunk to chunk
        part = slice(i, i + size)
        qi, ki, vi, bi = q[:, :, part], k[:, :, part], v[:, :, part], beta[:, :, part, None]
        total = decay[:, :, part].cumsum(-1)
        fade = torch.exp((total[..., :, None] - total[..., None, :]).masked_fill(~lower, -math.inf))
        # u = beta (v - what the state and the tokens before say), solved by (I - N)^-1 = (I + N)(I + N^2)(I + N^4)...
        n = -(bi * (ki @ ki.transpose(-1, -2)) * fade).tril(-1)
        solve, power, done = eye + n, n, 2
        while done < size:
            power = power @ power
            solve = solve + solve @ power
            done *= 2
        u = solve @ (bi * (vi - total[..., None].exp() * (ki @ state)))
        outs.append(total[..., None].exp() * (qi @ state) + ((qi @ ki.transpose(-1, -2)) * fade) @ u)
        left = (total[..., -1:] - total).exp()[..., None]
        state = total[..., -1, None, None].exp() * state + (ki * left).transpose(-1, -2) @ u
    out = torch.cat(outs, 2).transpose(1, 2)[real] * s["scale"]
    s["state"][s["slots"].long()] = state
    return {"out": out.to(s["out"].dtype), "state": s["state"]}


def _run_sample(s):
    if own:
        import bit_gemv_gb300 as nt
        nt.ninfer_sample(s["logits"], s["random"], temperature=s["temperature"], top_k=s["top_k"], top_p=s["top_p"],
                         min_p=s["min_p"], out=s["tokens"], logprobs=s["logprobs"])
        return {"tokens": s["tokens"], "logprobs": s["logprobs"]}
    column = lambda n: s[n].double()[:, None]  # noqa: E731
    x, order = torch.sort(s["logits"], descending=True, stable=True)
    greedy = column("temperature") <= 0
    rank = torch.arange(x.shape[1], device="cuda")[None, :]
    w = torch.exp((x.double() - x[:, :1].double()) / torch.where(greedy, 1.0, column("temperature")))
    w = w * torch.where(greedy, rank < 1, (s["top_k"][:, None] <= 0) | (rank < s["top_k"][:, None]))
    running = w.cumsum(1)
    w = w * ((running - w < column("top_p") * running[:, -1:]) & (w >= column("min_p")))
    w = torch.zeros_like(w).scatter_(1, order, w)
    running = w.cumsum(1)
    total = running[:, -1:]
    token = (running <= column("random") * total).sum(1, keepdim=True).clamp_(max=x.shape[1] - 1)
    return {"tokens": token[:, 0].int(), "logprobs": torch.log(w.gather(1, token) / total)[:, 0].float()}


# ------------------------------------------------------------------- work ---
def work(case):
    if case["op"] == "norm":
        row = BYTES[case["x"]] * (2 if case["gate"] else 1) + BYTES[case["out"]]
        row += 2 * BYTES[case["residual"]] if case["residual"] else 0
        return {"bytes": case["rows"] * case["cols"] * row + case["group"] * BYTES[case["weight"]], "flops": 0}
    if case["op"] == "rotary":
        row = (case["q_heads"] + case["kv_heads"]) * case["head_dim"] * 2 * BYTES[case["dtype"]]
        return {"bytes": case["tokens"] * (row + 4), "flops": 0}
    if case["op"] == "delta":
        tokens, size = sum(_news(case)), case["k_dim"] * case["v_dim"]
        row = 2 * case["k_heads"] * case["k_dim"] * BYTES[case["dtype"]] + 8 * case["v_heads"]
        row += case["v_heads"] * case["v_dim"] * (BYTES[case["dtype"]] + BYTES[case["out"]])
        return {"bytes": tokens * row + 4 * case["v_heads"] * size * (2 * case["requests"] - case["fresh"]),
                "flops": 6 * tokens * case["v_heads"] * size}
    return {"bytes": case["rows"] * (case["vocab"] * BYTES[case["dtype"]] + 28), "flops": 0}


# ------------------------------------------------------------------ exact ---
def exact(case, seed):
    """The definitions in 64 bits; whole numbers have no such value."""
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary, "delta": _exact_delta, "sample": _exact_sample}[case["op"]](s)


def _exact_norm(s):
    x = s["x"].double()
    total = None
    if s["residual"] is not None:
        x += s["residual"].double()
        total = x.clone()
    for g in range(0, x.shape[1], s["group"]):
        part = x[:, g:g + s["group"]]
        size = torch.sqrt((part * part).sum(1) / s["group"] + EPS)
        part /= size[:, None]
        part *= s["weight"].double()
    if s["gate"] is not None:
        x *= s["gate"].double() * torch.sigmoid(s["gate"].double())
    return {"out": x, "sum": total}


def _exact_rotary(s):
    turn = torch.polar(torch.ones((), dtype=torch.float64, device="cuda"), s["positions"].double()[:, None] * s["radians"])
    n = s["rotary_dim"]

    def turned(x, weight):
        y = x.double()
        if weight is not None:
            y = y / torch.sqrt((y * y).sum(-1, keepdim=True) / y.shape[-1] + EPS) * weight.double()
        pairs = y[..., :n].unflatten(-1, (-1, 2)) if s["interleaved"] else y[..., :n].unflatten(-1, (2, -1)).transpose(-1, -2)
        z = torch.view_as_real(torch.view_as_complex(pairs.contiguous()) * turn[:, None] * s["magnitude"])
        y[..., :n] = z.flatten(-2) if s["interleaved"] else z.transpose(-1, -2).flatten(-2)
        return y
    return {"q": turned(s["q"], s["q_weight"]), "k": turned(s["k"], s["k_weight"])}


def _exact_delta(s):
    """Token by token, the requests' tokens of one place together."""
    group = s["v"].shape[1] // s["k"].shape[1]
    slots, begin, count = s["slots"].long(), s["offsets"][:-1].long(), s["offsets"].diff().tolist()
    most = sorted(range(len(count)), key=lambda r: -count[r])
    state, out = s["state"].double(), torch.empty(s["v"].shape, dtype=torch.float64, device="cuda")
    state[slots[s["lengths"] == 0]] = 0
    order = torch.tensor(most, device="cuda")
    held, begin, alive = state[slots[order]], begin[order], len(most)

    def unit(x):
        x = x.double()
        return (x / torch.sqrt((x * x).sum(-1, keepdim=True) + s["eps"])).repeat_interleave(group, 1)
    for t in range(max(count)):
        while count[most[alive - 1]] <= t:
            alive -= 1
        at, now = begin[:alive] + t, held[:alive]
        q, k = unit(s["q"][at]), unit(s["k"][at])
        now *= torch.exp(s["log_decay"][at].double())[..., None, None]
        u = s["beta"][at].double()[..., None] * (s["v"][at].double() - torch.einsum("rhkv,rhk->rhv", now, k))
        now += k[..., :, None] * u[..., None, :]
        out[at] = torch.einsum("rhkv,rhk->rhv", now, q) * s["scale"]
    state[slots[order]] = held
    return {"out": out, "state": state}


def _exact_sample(s):
    found = []
    for b in range(len(s["random"])):
        x = s["logits"][b].double().cpu().numpy()
        t, k, p, least = float(s["temperature"][b]), int(s["top_k"][b]), float(s["top_p"][b]), float(s["min_p"][b])
        if t <= 0:
            found.append(0.0)
            continue
        order = np.argsort(-x, kind="stable")
        w = np.exp((x[order] - x.max()) / t)
        if k > 0:
            w = w[:k]
        reached = np.cumsum(w) >= p * w.sum()
        w = w[:int(np.argmax(reached)) + 1] if p < 1 and reached.any() else w
        w = w[w >= least]
        kept = order[:len(w)]
        by_index = np.argsort(kept)
        running = np.cumsum(w[by_index])
        at = min(int(np.searchsorted(running, float(s["random"][b]) * running[-1], side="right")), len(w) - 1)
        found.append(math.log(w[by_index[at]] / running[-1]))
    return {"tokens": None, "logprobs": torch.tensor(found, dtype=torch.float64, device="cuda")}
