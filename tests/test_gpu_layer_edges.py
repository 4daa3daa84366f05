"""Operators of a layer's step on the GPU where they went, or could go, wrong; against their fp64 definitions and against
themselves. Bounds as in test_gpu_layer.py unless derived here."""
import numpy as np
import pytest
import torch

import bit_gemv_gb300 as nt
from oracle import layer as ol
from test_gpu_layer import DEV, HALF, TORCH, check_sample, delta_case, f32, f64, i32, near, randn, run_delta

pytestmark = pytest.mark.gpu


# ----------------------------------------------------------------- sample ---
@pytest.mark.parametrize("rows,vocab,dtype", [(1, 248320, "f32"), (17, 248320, "f32"), (64, 248320, "f32"), (120, 60000, "bf16"), (300, 33000, "f32"),
                                              (700, 20000, "f32"), (40, 4099, "f16"), (9, 8195, "bf16")])
def test_sample_ctas_of_a_row_that_begin_late(rows, vocab, dtype):
    """Rows of two to sixteen CTAs, more of them than fit on the GPU at once and behind a kernel that leaves its SMs one by one: the same
    tokens each time, and the largest logit's for greedy rows."""
    g = torch.Generator("cuda").manual_seed(vocab + rows)
    x = (torch.randn(rows, vocab, generator=g, device=DEV) * 2).to(TORCH[dtype])
    random = torch.rand(rows, generator=g, device=DEV)
    temperature, p = torch.ones(rows, device=DEV), torch.full((rows,), 0.9, device=DEV)
    temperature[::3] = 0
    largest = x.float().max(1).values[::3]
    y, first = torch.randn(rows, vocab, generator=g, device=DEV), None
    for _ in range(20):
        nt.ninfer_norm(y)           # CTAs of long rows end at different times
        tokens = nt.ninfer_sample(x, random, temperature=temperature, top_p=p)
        if first is None:
            first = tokens
            assert torch.equal(x.float()[::3].gather(1, tokens[::3, None].long())[:, 0], largest)
        assert torch.equal(tokens, first)


def test_sample_least_temperatures():
    """Logits as small as their temperature, down to the least numbers: 2^-119 and all temperatures below it give the same, by the definition."""
    rng = np.random.default_rng(41)
    x = randn(rng, (6, 3000), "f32", 2.0 ** -118)
    random = rng.random(6).tolist()
    for controls in ({}, dict(top_p=[0.8] * 6), dict(top_k=[9] * 6), dict(min_p=[0.05] * 6)):
        tokens = check_sample(x, random, temperature=[2.0 ** -119] * 6, **controls)
        for t in (1e-36, 2e-38, 1e-45):
            args = {n: (i32 if n == "top_k" else f32)(c) for n, c in controls.items()}
            assert nt.ninfer_sample(x, f32(random), temperature=f32([t] * 6), **args).tolist() == tokens
    assert len(set(tokens)) > 1


# ------------------------------------------------------------ gated delta ---
def test_gated_delta_single_tokens_take_no_workspace():
    """Without offsets nothing is allocated beside the result, and a size that no workspace could have is no matter."""
    case = delta_case(np.random.default_rng(1), 40, 40, 2, 6, 64, 64, "bf16")
    out = nt.ninfer_gated_delta(**case)
    count = lambda: torch.cuda.memory_stats()["allocation.all.allocated"]  # noqa: E731
    before = count()
    nt.ninfer_gated_delta(**case, out=out)
    assert count() == before
    nt.ninfer_gated_delta(**case)
    assert count() == before + 1
    nt.ninfer_gated_delta(**case, offsets=i32([0, 40]), out=out)
    assert count() >= before + 2        # a prompt's, and the offsets


# few states (results by warps of their own, with a ninth warp and without) and more than SMs (32 and 64 columns a CTA)
INSTANCES = [(1, 2, 64, 48, "bf16"), (1, 2, 128, 40, "bf16"), (1, 2, 96, 32, "f32"), (2, 4, 256, 16, "f16"), (8, 160, 128, 24, "bf16"),
             (4, 160, 96, 24, "f32"), (2, 160, 256, 16, "bf16"), (1, 160, 256, 8, "f32")]


@pytest.mark.parametrize("k_heads,v_heads,dk,dv,dtype", INSTANCES)
@pytest.mark.parametrize("widest", [0, 20, 40, 60])
def test_gated_delta_prompts_of_unequal_sizes(k_heads, v_heads, dk, dv, dtype, widest):
    """Without norms: queries, and keys with the betas that suit them, whose sizes differ by up to 2^widest among the tokens of a chunk. A
    token's result is as exact as its own query and the state allow."""
    if dtype == "f16" and widest > 20:
        widest = 20             # its exponents
    rng = np.random.default_rng(dk + widest)
    case = delta_case(rng, 90, 2, k_heads, v_heads, dk, dv, dtype, 2)
    sizes = lambda: f32(2.0 ** -rng.integers(0, widest + 1, (90, 1, 1)))  # noqa: E731
    for n, most in (("q", 1.0), ("k", 4.0)):
        size = sizes()
        case[n] = (case[n].float() * dk ** -0.5 * size * (most if dtype != "f16" else 1)).to(TORCH[dtype])
    norm = case["k"].float().square().sum(-1).repeat_interleave(v_heads // k_heads, 1)
    case["beta"] = torch.minimum(case["beta"], 1 / norm)
    run_delta(case, "f32", offsets=[0, 58, 90], norm_eps=None)


@pytest.mark.parametrize("dk,dtype", [(128, "bf16"), (96, "f32"), (256, "f32")])
@pytest.mark.parametrize("v_heads", [2, 160])
def test_gated_delta_prompts_with_small_queries(dk, v_heads, dtype):
    """A query's size has no part in the bits of its result: queries times powers of two give results times those, bit by bit."""
    rng = np.random.default_rng(dk)
    case = delta_case(rng, 100, 1, 1, v_heads, dk, 16, dtype, 1)
    case["k"] = case["k"] * dk ** -0.5
    size = torch.exp2(-f32(rng.integers(0, 50, 100))).float()
    state = case["state"].clone()
    out = nt.ninfer_gated_delta(**case, offsets=i32([0, 100]), out_dtype=torch.float32)
    case["state"], case["q"] = state, (case["q"].float() * size[:, None, None]).to(TORCH[dtype])
    small = nt.ninfer_gated_delta(**case, offsets=i32([0, 100]), out_dtype=torch.float32)
    assert torch.equal(small, out * size[:, None, None])


def check_finite_parts(case, offsets, norm_eps=1e-6, out_dtype="f32", **kw):
    """What is finite by the definition is right, and nothing else is finite."""
    tokens, v_heads, dv = case["v"].shape
    args = [f64(case[n]) for n in ("q", "k", "v", "log_decay", "beta", "state")]
    with np.errstate(all="ignore"):
        want, state, out_bound, bound = ol.gated_delta(*args, offsets, range(len(offsets) - 1), None, case["q"].shape[2] ** -0.5, norm_eps,
                                                       2.0 ** -23, 2.0 ** -39)
    out = nt.ninfer_gated_delta(**case, offsets=i32(offsets), norm_eps=norm_eps, out_dtype=TORCH[out_dtype], **kw)
    for got, want, bound, half in ((f64(out), want, out_bound, HALF[out_dtype]), (f64(case["state"]), state, bound, HALF["f32"])):
        live = np.isfinite(want)
        assert np.array_equal(np.isfinite(got), live), (np.argwhere(np.isfinite(got) != live)[:5], live.mean())
        assert (np.abs(got - want)[live] <= bound[live] + half * np.abs(want[live]) + 1e-40).all()
    return out


@pytest.mark.parametrize("k_heads,v_heads,dk,dv,dtype", INSTANCES)
@pytest.mark.parametrize("norm_eps", [1e-6, None])
def test_gated_delta_non_finite_values_reach_no_earlier_token(k_heads, v_heads, dk, dv, dtype, norm_eps):
    """An infinity or NaN at a token of a prompt changes that token and the later ones of its columns, heads and request, and nothing before
    or beside them, wherever it lies among the 32 tokens of a chunk."""
    rng = np.random.default_rng(dk + v_heads)
    offsets = [0, 67, 75, 110]
    clean = delta_case(rng, 110, 3, k_heads, v_heads, dk, dv, dtype, 3)
    for n in ("q", "k"):
        clean[n] = (clean[n] * dk ** -0.5).contiguous()
    for i, n in enumerate(("q", "k", "v", "log_decay", "beta", "state")):
        for value in (float("nan"), float("inf"), -float("inf"))[i % 3 if v_heads > 99 else 0:i % 3 + 1 if v_heads > 99 else 3]:
            case = {m: t.clone() for m, t in clean.items()}
            if n == "state":
                case[n][1, v_heads - 1, dk // 2, dv - 3] = value
            else:
                for t in (rng.integers(0, 16), 16 + rng.integers(0, 16), 32 + rng.integers(0, 35), 67, 109)[rng.integers(0, 2)::2]:
                    at = case[n][int(t), int(rng.integers(0, case[n].shape[1]))]
                    if n in ("q", "k", "v"):
                        at[int(rng.integers(0, at.shape[0]))] = value
                    else:
                        at.fill_(value)
            check_finite_parts(case, offsets, norm_eps)


def test_gated_delta_non_finite_values_of_many_tokens():
    """Whole columns of values, all decays, a prompt's first and last tokens."""
    rng = np.random.default_rng(3)
    nan, inf = float("nan"), float("inf")
    for dk, dtype in ((128, "bf16"), (256, "f32")):
        for v_heads in (2, 160):
            case = delta_case(rng, 70, 1, 1, v_heads, dk, 24, dtype, 1)
            case["v"][:, 0, 3], case["v"][69, 1, 5], case["v"][0, 1, 6] = inf, nan, -inf
            case["v"][40, 1, 7], case["v"][33, 1, 7] = nan, inf
            case["beta"][64:, 1] = nan
            check_finite_parts(case, [0, 70])
            case = delta_case(rng, 70, 1, 1, v_heads, dk, 24, dtype, 1)
            case["q"][::2, 0, 1] = nan
            case["log_decay"].fill_(-inf)
            check_finite_parts(case, [0, 70])


@pytest.mark.parametrize("k_heads,v_heads,dk,dv,dtype", [(4, 8, 128, 128, "bf16"), (2, 4, 64, 64, "f16"), (2, 4, 96, 80, "f32"), (1, 6, 256, 48, "bf16"),
                                                         (1, 6, 256, 72, "f32")])
def test_gated_delta_a_request_alone_and_among_others(k_heads, v_heads, dk, dv, dtype):
    """The number of requests picks the columns of a CTA and who makes the results; no bit of a request's results depends on it."""
    rng = np.random.default_rng(dk + dv)
    lengths = rng.integers(1, 140, 90)
    offsets = np.concatenate([[0], np.cumsum(lengths)])
    case = delta_case(rng, offsets[-1], 90, k_heads, v_heads, dk, dv, dtype, 90)
    for norm_eps in (1e-6, None):
        if norm_eps is None:
            case["k"] = case["k"] * dk ** -0.5
        state = case["state"].clone()
        out = nt.ninfer_gated_delta(**{**case, "state": state}, offsets=i32(offsets), norm_eps=norm_eps)
        for some in ([0], [17], [89], [3, 50], list(range(12, 24)), list(range(40, 70))):
            part = {n: torch.cat([case[n][offsets[r]:offsets[r + 1]] for r in some]) for n in ("q", "k", "v", "log_decay", "beta")}
            s, o = case["state"][some].clone(), np.concatenate([[0], np.cumsum(lengths[some])])
            got = nt.ninfer_gated_delta(**part, state=s, offsets=i32(o), norm_eps=norm_eps)
            assert torch.equal(got, torch.cat([out[offsets[r]:offsets[r + 1]] for r in some])) and torch.equal(s, state[some])


@pytest.mark.parametrize("dk,dtype", [(64, "bf16"), (128, "f32"), (256, "f16")])
def test_gated_delta_requests_in_any_order_of_their_tokens(dk, dtype):
    """Offsets that fall begin again further ahead; requests without tokens lie between."""
    rng = np.random.default_rng(dk)
    for offsets in ([64, 100, 0, 64], [128, 256, 0, 128], [200, 231, 100, 200, 33, 100, 0, 33], [161, 162, 96, 161, 0, 32, 32, 64, 64, 96], [70, 5000, -3, 70]):
        case = delta_case(rng, max(min(max(offsets), 300), 1), len(offsets) - 1, 1, 2, dk, 24, dtype)
        run_delta(case, offsets=offsets)


@pytest.mark.parametrize("dk,dtype,v_heads", [(128, "bf16", 4), (96, "f32", 4), (256, "f16", 160), (128, "f32", 160)])
def test_gated_delta_prompts_cut_at_chunks(dk, dtype, v_heads):
    """A prompt in several calls, cut at multiples of 32 tokens, gives the bits of one call, whose workspace grows with it."""
    rng = np.random.default_rng(dk)
    case = delta_case(rng, 203, 1, 2, v_heads, dk, 40, dtype, 1)
    state, parts = case["state"].clone(), []
    for a, b in ((0, 32), (32, 128), (128, 203)):
        part = {n: case[n][a:b] for n in ("q", "k", "v", "log_decay", "beta")}
        parts.append(nt.ninfer_gated_delta(**part, state=state, offsets=i32([0, b - a]), lengths=i32([a]), norm_eps=1e-6))
    whole = nt.ninfer_gated_delta(**case, offsets=i32([0, 203]), lengths=i32([0]), norm_eps=1e-6)
    assert torch.equal(torch.cat(parts), whole) and torch.equal(state, case["state"])


@pytest.mark.parametrize("dk,dv,dtype,requests", [(128, 128, "bf16", 6), (64, 40, "f32", 6), (256, 72, "f16", 60), (96, 64, "bf16", 200)])
def test_gated_delta_single_tokens_of_non_finite_values(dk, dv, dtype, requests):
    """Infinities and NaN of a request's token stay with its heads and columns."""
    rng = np.random.default_rng(dk)
    clean = delta_case(rng, requests, requests, 2, 4, dk, dv, dtype, requests)
    for n in ("q", "k", "v", "log_decay", "beta", "state"):
        for value in (float("nan"), float("inf"), -float("inf")):
            case = {m: t.clone() for m, t in clean.items()}
            r, h = int(rng.integers(0, requests)), int(rng.integers(0, case[n].shape[1]))
            if n == "state":
                case[n][r, h, dk - 1, dv // 2] = value
            elif n in ("q", "k", "v"):
                case[n][r, h, 3] = value
            else:
                case[n][r, h] = value
            with np.errstate(all="ignore"):
                want, state, out_bound, bound = ol.gated_delta(*(f64(case[m]) for m in ("q", "k", "v", "log_decay", "beta", "state")), range(requests + 1),
                                                               range(requests), None, dk ** -0.5, 1e-6, 2.0 ** -23)
            out = nt.ninfer_gated_delta(**case, norm_eps=1e-6, out_dtype=torch.float32)
            for got, want, bound in ((f64(out), want, out_bound), (f64(case["state"]), state, bound)):
                live = np.isfinite(want)
                assert np.array_equal(np.isfinite(got), live) and (np.abs(got - want)[live] <= bound[live] + HALF["f32"] * np.abs(want[live]) + 1e-40).all()


# ------------------------------------------------------------------- norm ---
@pytest.mark.parametrize("group", [128, 24, 512, 5, 33000])
def test_norm_gates_of_any_size(group):
    """z / (1 + e^-z) however far from 0, infinities and NaN as the formula has them. In units of 2^-24 the root of the squares' sum is off by 23
    (test_gpu_layer.py), the reciprocal root by 4, the exponential by 14, the reciprocal by 2, a sum and four products by one each: 48."""
    rng = np.random.default_rng(group)
    cols = group * max(1, 2048 // group)
    x = randn(rng, (8, cols))
    gate = f32(rng.uniform(-104, 104, (8, cols)))
    gate[1] = f32(rng.uniform(-89, -86, cols))
    gate[2] = f32(rng.standard_normal(cols) * 1e-3)
    gate[3, :5] = f32([1e30, -1e30, 0.0, -0.0, 3e38])
    for dtype in ("f32", "bf16"):
        xd, gd = x.to(TORCH[dtype]), gate.to(TORCH[dtype])
        _, want = ol.norm(f64(xd), None, f64(gd), None, group, 1e-5)
        near(f64(nt.ninfer_norm(xd, None, 1e-5, gate=gd, group=group, out_dtype=torch.float32)), want, 48 * 2.0 ** -24 * np.abs(want), "f32")
    gate[0, 0], gate[0, 1], gate[0, 2] = float("inf"), -float("inf"), float("nan")
    x[0, 0] = 1.0
    y = nt.ninfer_norm(x, None, 1e-5, gate=gate, group=group)
    assert y[0, 0] == float("inf") and y[0, 1:3].isnan().all() and y[0, 3:].isfinite().all()


# ------------------------------------------------------------------ views ---
def test_views_between_each_others_rows_are_taken():
    """Parts of one buffer that share no element, whatever their strides, and outputs that the documentation allows over inputs."""
    rng = np.random.default_rng(31)
    # norm: x, residual, gate, sum and out as columns of one buffer; rows of two strides between each other
    wide = randn(rng, (6, 5 * 64))
    x, r, g, s, o = (wide[:, i * 64:(i + 1) * 64] for i in range(5))
    want_s, want = ol.norm(f64(x), f64(r), f64(g))
    nt.ninfer_norm(x, residual=r, gate=g, sum=s, out=o)
    near(f64(o), want, 48 * 2.0 ** -24 * np.abs(want), "f32")
    near(f64(s), want_s, 2.0 ** -24 * np.abs(want_s), "f32")
    rows = randn(rng, (12, 64))
    even, third = rows[0:9:2], rows[1:12:4]                 # x at 0, 2, 4; out at 1, 5, 9
    before = rows.clone()
    nt.ninfer_norm(even[:3], out=third)
    assert torch.equal(third, nt.ninfer_norm(before[0:5:2]))
    third.copy_(before[1:12:4])
    assert torch.equal(rows, before)
    # rotary: queries and gates by turns in rows that end with keys, in place; heads before tokens
    q_heads, kv, dim = 4, 2, 64
    width = (2 * q_heads + kv) * dim
    buffer = randn(rng, (5, width))
    q, k = buffer[:, :2 * q_heads * dim].unflatten(1, (q_heads, 2 * dim))[:, :, :dim], buffer[:, 2 * q_heads * dim:].unflatten(1, (kv, dim))
    freq, positions = torch.from_numpy(nt.ninfer_rotary_frequencies(dim)[0]).to(DEV), i32(np.arange(5) * 7)
    gates = buffer[:, :2 * q_heads * dim].unflatten(1, (q_heads, 2 * dim))[:, :, dim:]
    kept, apart = gates.clone(), nt.ninfer_rotary(q.clone(), k.clone(), positions, freq)
    nt.ninfer_rotary(q, k, positions, freq, q_out=gates)     # the gates' places
    assert torch.equal(gates, apart[0]) and torch.equal(k, apart[1])
    gates.copy_(kept)
    turned = randn(rng, (q_heads + kv, 5, dim))
    qt, kt = turned[:q_heads].transpose(0, 1), turned[q_heads:].transpose(0, 1)
    apart = nt.ninfer_rotary(qt.clone(), kt.clone(), positions, freq)
    nt.ninfer_rotary(qt, kt, positions, freq)
    assert torch.equal(qt, apart[0]) and torch.equal(kt, apart[1])
    # gated delta: states between which the results lie, and results in the values' place
    for tokens, offsets in ((3, None), (70, i32([0, 40, 65, 70]))):
        case = delta_case(rng, tokens, 3, 1, 2, 64, 32, "f32", 3)
        state = case["state"].clone()
        want = nt.ninfer_gated_delta(**{**case, "state": state}, offsets=offsets)
        pool = torch.zeros(3, 2 * 64 * 32 + tokens * 64, device=DEV)
        pool[:, :4096] = case["state"].flatten(1)
        got = nt.ninfer_gated_delta(**{**case, "state": pool[:, :4096].unflatten(1, (2, 64, 32))}, offsets=offsets, out=pool[1, 4096:].view(tokens, 2, 32))
        assert torch.equal(got, want) and torch.equal(pool[:, :4096], state.flatten(1)) and not pool[0, 4096:].any() and not pool[2, 4096:].any()
        values = case["v"].contiguous()
        state = case["state"].clone()
        assert nt.ninfer_gated_delta(**{**case, "state": state, "v": values}, offsets=offsets, out=values) is values
        assert torch.equal(values, want)
    # sampling: results in the controls' place
    x, random, k = randn(rng, (9, 60000)), f32(rng.random(9)), i32([0, 3, 50, 0, 7, 0, 0, 1, 2000])
    logprobs = torch.empty(9, device=DEV)
    tokens = nt.ninfer_sample(x, random, top_k=k, logprobs=logprobs)
    nt.ninfer_sample(x, random, top_k=k, out=k, logprobs=random)
    assert torch.equal(k, tokens) and torch.equal(random, logprobs)


@pytest.mark.parametrize("dk,dv,v_heads,dtype", [(128, 128, 4, "bf16"), (64, 40, 4, "f16"), (128, 72, 160, "bf16"), (256, 24, 160, "f32"), (96, 48, 6, "f32")])
def test_gated_delta_results_in_the_values_place(dk, dv, v_heads, dtype):
    rng = np.random.default_rng(dk + dv)
    for tokens, offsets in ((3, None), (400, i32([0, 340, 341, 400]))):
        case = delta_case(rng, tokens, 3, 2, v_heads, dk, dv, dtype, 3)
        state, values = case["state"].clone(), case["v"].contiguous()
        want = nt.ninfer_gated_delta(**{**case, "state": state}, offsets=offsets)
        nt.ninfer_gated_delta(**{**case, "v": values}, offsets=offsets, out=values)
        # bit by bit: without norms the states grow beyond all numbers, and NaN is no NaN's equal
        same = lambda a, b: torch.equal(a.view(torch.int16), b.view(torch.int16))  # noqa: E731
        assert same(values, want) and same(case["state"], state)
