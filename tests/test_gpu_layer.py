"""Operators of a layer's step on the GPU against their fp64 definitions.

Bounds, fixed from the number formats (h: half a step of the output's format):
- norm: the sum is one fp32 rounding, then the output's. A square sum's terms hold three roundings each and go through at
  most 32 additions in a thread and 10 between threads, so that its root is off by 23 2^-24; root, quotient, three
  products, weight + offset and the gate (expf within 2 units, sum, quotient, product) add at most 16: 40 2^-24.
- rotary: the fraction of a turn is a float in [-1, 1] half turns (2^-25), sincospif within 2^-23, four roundings, and a
  norm within 20 2^-24: (|a| + |b|) magnitude 2^-20.
- gated delta: oracle.layer.gated_delta's own bound, with roundings of 2^-23 (fp32 sums, operands of two binary16 terms), and for
  several tokens a request binary16's least step, 2^-24, where a column's largest operand is at 2^13 and more: half of it is 2^-39.
- sample: a weight is off by 2^-30 of itself and 2^-43 of the largest, sums are exact: the token is the oracle's wherever
  its nearest border is 2^-28 away. logprob: 2^-22 of itself and of 1, two fp32 functions.
"""
import math

import numpy as np
import pytest
import torch

import bit_gemv_gb300 as nt
from oracle import layer as ol

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}
HALF = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def f32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.float32)).to(DEV)


def randn(rng, shape, dtype="f32", scale=1.0):
    return f32(rng.standard_normal(shape) * scale).to(TORCH[dtype])


def near(got, want, bound, dtype):
    """Within the bound and half a step of the format (2^-25 absolute where float16 has no smaller one)."""
    assert np.array_equal(np.isnan(got), np.isnan(want))
    ok = np.abs(got - want) <= bound + HALF[dtype] * np.abs(want) + (2.0 ** -25 if dtype == "f16" else 1e-40)
    assert (ok | np.isnan(want)).all(), np.abs(got - want).max()


# ------------------------------------------------------------------- norm ---
@pytest.mark.parametrize("rows,cols,group", [
    (1, 5120, None), (3, 8, None), (2, 1, None), (5, 7, None), (7, 1000, None), (2, 8200, None), (3, 16385, None), (2, 32768, None),
    (2, 40001, None), (9, 48, 8), (4, 96, 24), (33, 6 * 64, 64), (5, 12 * 128, 128), (4, 3 * 160, 160), (3, 5 * 256, 256), (3, 2 * 264, 264),
    (5, 35, 5), (1000, 512, 128)])
@pytest.mark.parametrize("x,residual,out", [("f32", "f32", "bf16"), ("bf16", "bf16", "f16"), ("f16", "f32", "f32"), ("bf16", None, "bf16"),
                                            ("f32", "f16", "f32")])
def test_norm(rows, cols, group, x, residual, out):
    rng = np.random.default_rng(rows * 1000 + cols)
    xd, w = randn(rng, (rows, cols), x), randn(rng, (group or cols,), "bf16" if cols % 2 else "f32")
    rd = randn(rng, (rows, cols), residual, 4) if residual else None
    gate = randn(rng, (rows, 2 * cols), x, 3)[:, cols:] if group else None
    sd = torch.full((rows, cols), 7.0, device=DEV).to(TORCH[residual]) if residual else None
    y = nt.ninfer_norm(xd, w, 1e-5, residual=rd, sum=sd, gate=gate, group=group, weight_offset=1.0, out_dtype=TORCH[out])
    s, want = ol.norm(f64(xd), f64(rd) if residual else None, f64(gate) if group else None, f64(w), group, 1e-5, 1.0)
    assert y.dtype is TORCH[out]
    near(f64(y), want, 40 * 2.0 ** -24 * np.abs(want), out)
    if residual:
        near(f64(sd), s, 2.0 ** -24 * np.abs(s), residual)


def test_norm_in_place_strided_and_plain():
    """The residual stream updated in place, x replaced by its norm, rows of a wider tensor; no weight; huge and zero rows."""
    rng = np.random.default_rng(1)
    for cols in (256, 5120, 77, 40001):
        wide = randn(rng, (6, cols + 24), "bf16")
        x, stream = wide[:, 8:8 + cols], randn(rng, (6, cols))
        x[2], stream[2] = 0, 0
        stream[3] *= 1e15
        s, want = ol.norm(f64(x), f64(stream), None, None, None, 1e-6)
        kept = wide.clone()
        assert nt.ninfer_norm(x, None, 1e-6, residual=stream, sum=stream, out=x) is x
        near(f64(x), want, 40 * 2.0 ** -24 * np.abs(want), "bf16")
        near(f64(stream), s, 2.0 ** -24 * np.abs(s), "f32")
        assert torch.equal(wide[:, :8], kept[:, :8]) and torch.equal(wide[:, 8 + cols:], kept[:, 8 + cols:])
        assert not x[2].any()


def test_norm_keeps_nan_and_infinity_to_their_group():
    x = torch.ones(4, 512, device=DEV)
    x[1, 130], x[2, 300] = float("nan"), float("inf")
    y = nt.ninfer_norm(x, group=128)
    bad = torch.zeros(4, 512, dtype=torch.bool, device=DEV)
    bad[1, 128:256], bad[2, 300] = True, True
    assert torch.equal(torch.isnan(y), bad)
    assert not y[2, 256:300].any() and (y[0] == y[3]).all()


# ----------------------------------------------------------------- rotary ---
def rotary_case(rng, tokens, q_heads, kv_heads, dim, dtype):
    rows = randn(rng, (tokens, q_heads + 2 * kv_heads + 1, dim), dtype)
    return rows, rows[:, 1:1 + q_heads], rows[:, 1 + q_heads:1 + q_heads + kv_heads]


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,q_heads,kv_heads,dim,rotary_dim,dtype", [
    (1, 1, 1, 8, 8, "f32"), (3, 24, 4, 256, 64, "bf16"), (5, 8, 8, 128, 128, "f16"), (7, 6, 2, 80, 80, "bf16"), (4, 40, 5, 96, 24, "f32"),
    (2, 3, 1, 192, 192, "f32"), (6, 16, 2, 64, 2, "bf16"), (3, 100, 4, 48, 20, "f32"), (70, 2, 1, 72, 40, "f16"), (5, 4, 4, 256, 256, "f32")])
def test_rotary(tokens, q_heads, kv_heads, dim, rotary_dim, dtype, interleaved):
    rng = np.random.default_rng(dim + tokens)
    rows, q, k = rotary_case(rng, tokens, q_heads, kv_heads, dim, dtype)
    positions = rng.integers(0, 2 ** 31, tokens)
    positions[0] = 0
    if tokens > 2:
        positions[1], positions[2] = 2 ** 31 - 1, -5
    table, magnitude = nt.ninfer_rotary_frequencies(rotary_dim, 1e4, "dimensions", factor=4.0, context=8192.0)
    turns = table.view(np.uint64)
    weights = [None, None] if tokens % 2 else [randn(rng, (dim,), dtype) for _ in range(2)]
    for w, name, x in ((weights[0], "q", q), (weights[1], "k", k)):
        want = ol.rotary(f64(x), positions, turns, magnitude, interleaved, f64(w) if w is not None else None, 1e-5, 1.0)
        size = ol.rotary(f64(x), np.minimum(positions, 0), turns, magnitude, interleaved, f64(w) if w is not None else None, 1e-5, 1.0)
        half = rotary_dim // 2
        bound = np.abs(size)
        if interleaved:
            pair = bound[..., :rotary_dim].reshape(*bound.shape[:2], half, 2)
            bound[..., :rotary_dim] = np.repeat(pair.sum(-1), 2, -1)
        else:
            bound[..., :rotary_dim] = np.tile(bound[..., :half] + bound[..., half:rotary_dim], 2)
        if name == "q":
            q_want, q_bound = want, bound * 2.0 ** -20
        else:
            k_want, k_bound = want, bound * 2.0 ** -20
    args = dict(interleaved=interleaved, q_weight=weights[0], k_weight=weights[1], eps=1e-5, weight_offset=1.0)
    freq = torch.from_numpy(table).to(DEV)
    q_out, k_out = torch.full_like(q.contiguous(), 9.0), torch.full_like(k.contiguous(), 9.0)
    before = rows.clone()
    nt.ninfer_rotary(q, k, i32(positions), freq, magnitude, q_out=q_out, k_out=k_out, **args)
    assert torch.equal(rows, before)
    for got, want, bound in ((q_out, q_want, q_bound), (k_out, k_want, k_bound)):
        left = np.isnan(want)
        assert (f64(got)[left] == 9).all()
        near(np.where(left, np.nan, f64(got)), want, np.where(left, 0, bound), dtype)
    # in place: the same bits, nothing else of the rows, left-out tokens as they were
    nt.ninfer_rotary(q, k, i32(positions), freq, magnitude, **args)
    here = torch.from_numpy(positions >= 0).to(DEV)
    assert torch.equal(q[here], q_out[here]) and torch.equal(k[here], k_out[here]) and torch.equal(rows[~here], before[~here])
    assert torch.equal(rows[:, 0], before[:, 0]) and torch.equal(rows[:, 1 + q_heads + kv_heads:], before[:, 1 + q_heads + kv_heads:])


def test_rotary_queries_alone_and_one_norm():
    rng = np.random.default_rng(3)
    _, q, k = rotary_case(rng, 9, 4, 2, 64, "f32")
    table, _ = nt.ninfer_rotary_frequencies(64, 1e4)
    freq, positions, w = torch.from_numpy(table).to(DEV), i32(np.arange(9) * 1000), randn(rng, (64,), "bf16")
    both = nt.ninfer_rotary(q, k, positions, freq, q_out=torch.empty_like(q), k_out=torch.empty_like(k), k_weight=w)
    alone, none = nt.ninfer_rotary(q, None, positions, freq, q_out=torch.empty_like(q))
    assert none is None and torch.equal(both[0], alone)
    want = ol.rotary(f64(k), np.arange(9) * 1000, table.view(np.uint64), 1.0, False, f64(w))
    near(f64(both[1]), want, 2.0 ** -20 * (np.abs(f64(w)).max() * 8), "f32")


# ------------------------------------------------------------ gated delta ---
def delta_case(rng, tokens, requests, k_heads, v_heads, dk, dv, dtype, slots=None):
    width = 2 * k_heads * dk
    rows = randn(rng, (tokens, width + v_heads * dv + 8), dtype)
    split = lambda a, n: a.unflatten(1, (n, -1))  # noqa: E731
    return dict(q=split(rows[:, :width // 2], k_heads), k=split(rows[:, width // 2:width], k_heads), v=split(rows[:, width:width + v_heads * dv], v_heads),
                log_decay=f32(-np.exp(rng.standard_normal((tokens, v_heads + 3)) - 3))[:, :v_heads],
                beta=f32(1 / (1 + np.exp(-rng.standard_normal((tokens, v_heads))))), state=randn(rng, (slots or requests + 2, v_heads, dk, dv), "f32", 0.5))


def run_delta(case, out_dtype="f32", offsets=None, slots=None, lengths=None, norm_eps=1e-6, unit=2.0 ** -23, **kw):
    tokens, v_heads, dv = case["v"].shape
    dk = case["q"].shape[2]
    n = tokens if offsets is None else len(offsets) - 1
    cut = np.arange(n + 1) if offsets is None else np.clip(offsets, 0, tokens)
    held = list(range(n)) if slots is None else slots
    want, state, out_bound, bound = ol.gated_delta(*(f64(case[x]) for x in ("q", "k", "v", "log_decay", "beta", "state")), cut, held,
                                                   lengths, dk ** -0.5, norm_eps, unit, 2.0 ** -39 if offsets is not None else 0.0)
    out = torch.full((tokens, v_heads, dv), 5.0, device=DEV).to(TORCH[out_dtype])
    before = case["state"].clone()
    nt.ninfer_gated_delta(**case, offsets=None if offsets is None else i32(offsets), slots=None if slots is None else i32(slots),
                          lengths=None if lengths is None else i32(lengths), norm_eps=norm_eps, out=out, **kw)
    got = f64(out)
    assert (got[np.isnan(want)] == 5).all()
    near(np.where(np.isnan(want), np.nan, got), want, out_bound, out_dtype)
    near(f64(case["state"]), state, bound, "f32")
    touched = {int(s) for s, b, e in zip(held, cut[:-1], cut[1:]) if e > b}
    for s in set(range(len(before))) - touched:
        assert torch.equal(case["state"][s], before[s])
    return out


SHAPES = [(1, 1, 8, 8), (2, 4, 64, 64), (1, 3, 128, 128), (2, 2, 96, 64), (1, 2, 128, 256), (1, 2, 256, 128), (2, 6, 48, 80), (1, 1, 256, 256),
          (4, 4, 16, 24), (1, 2, 136, 40)]


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("k_heads,v_heads,dk,dv", SHAPES)
def test_gated_delta_one_token_each(k_heads, v_heads, dk, dv, dtype, out):
    rng = np.random.default_rng(dk + dv)
    run_delta(delta_case(rng, 3, 3, k_heads, v_heads, dk, dv, dtype), out)
    run_delta(delta_case(rng, 5, 5, k_heads, v_heads, dk, dv, dtype, 9), out, slots=[7, -1, 0, 3, 8], lengths=[4, 1, 0, -3, 1], norm_eps=None)


def test_gated_delta_a_batch_of_single_tokens():
    """Enough requests for whole rows of a state a CTA."""
    rng = np.random.default_rng(2)
    run_delta(delta_case(rng, 160, 160, 1, 2, 128, 128, "bf16"), "bf16", slots=rng.permutation(162)[:160].tolist())
    run_delta(delta_case(rng, 320, 320, 1, 1, 40, 96, "f32"))


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("k_heads,v_heads,dk,dv", SHAPES)
def test_gated_delta_ragged(k_heads, v_heads, dk, dv, dtype, out):
    rng = np.random.default_rng(dk * 3 + dv)
    counts = [1, 0, 37, 64, 5, 130, 16]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    case = delta_case(rng, offsets[-1] + 3, 7, k_heads, v_heads, dk, dv, dtype, 10)
    run_delta(case, out, offsets=offsets, slots=[3, 5, 9, -1, 0, 2, 1], lengths=[5, 0, 0, 7, 1, 0, 9])


@pytest.mark.parametrize("dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f16", "f32")])
@pytest.mark.parametrize("dk", [64, 96, 128, 256])
def test_gated_delta_ragged_many_heads(dk, dtype, out):
    """More states than SMs: 32 or 64 columns a CTA, the last of them with eight."""
    rng = np.random.default_rng(dk)
    counts = [70, 1, 0, 33, 128, 6]
    offsets = np.concatenate([[0], np.cumsum(counts)])
    case = delta_case(rng, offsets[-1], 6, 4, 28, dk, 72, dtype, 7)
    run_delta(case, out, offsets=offsets, slots=[6, 3, 1, 0, 2, 5], lengths=[0, 3, 1, 0, 5, 0])


@pytest.mark.parametrize("dv", [8, 16, 40, 48, 104, 152, 248])
@pytest.mark.parametrize("dk,dtype", [(128, "bf16"), (128, "f32"), (96, "bf16"), (256, "f16"), (256, "f32")])
def test_gated_delta_columns_of_a_prompt(dk, dv, dtype):
    """16 columns a CTA, and what is left of them for the last."""
    rng = np.random.default_rng(dk + dv)
    run_delta(delta_case(rng, 230, 1, 1, 2, dk, dv, dtype), "f32" if dv % 16 else dtype, offsets=[0, 227])


@pytest.mark.parametrize("v_heads,dv", [(36, 128), (36, 104), (48, 128), (48, 104), (48, 72), (152, 48), (152, 24), (150, 40)])
@pytest.mark.parametrize("dk,dtype", [(128, "bf16"), (128, "f32"), (64, "f16"), (96, "f32"), (256, "bf16"), (256, "f32")])
def test_gated_delta_columns_of_many_heads(dk, v_heads, dv, dtype):
    """32 and 48 columns a CTA where those fill the SMs, one to three pairs of warps in the last."""
    rng = np.random.default_rng(dk + dv + v_heads)
    run_delta(delta_case(rng, 140, 1, 2, v_heads, dk, dv, dtype), dtype, offsets=[0, 139])


def test_gated_delta_offsets_of_any_value():
    rng = np.random.default_rng(7)
    for offsets in ([-5, 3, 3, 9, 40], [0, 2 ** 31 - 1, 7, 7, -2 ** 31], [30, 30, 0, 5, 5], [9, 12, 4, 4, 9]):
        case = delta_case(rng, 12, 4, 1, 2, 64, 64, "bf16")
        run_delta(case, offsets=offsets)


def test_gated_delta_bad_slots():
    rng = np.random.default_rng(8)
    for offsets in (None, [0, 2, 3, 6]):
        case = delta_case(rng, 3 if offsets is None else 6, 3, 1, 2, 64, 32, "f32", 4)
        status = torch.zeros(1, dtype=torch.int32, device=DEV)
        run_delta(case, offsets=offsets, slots=[1, 4, 2 ** 31 - 1], status=status)
        assert int(status) == nt.DELTA_BAD_SLOT
        status.zero_()
        run_delta(case, offsets=offsets, slots=[1, -1, 2], status=status)
        assert int(status) == 0


def test_gated_delta_parts_make_the_whole():
    """A prompt at once, in two parts, and its last tokens one by one: the same within the bounds of each."""
    rng = np.random.default_rng(9)
    case = delta_case(rng, 150, 1, 2, 4, 128, 128, "bf16", 1)
    whole = case["state"].clone()
    out = run_delta({**case, "state": whole}, offsets=[0, 150], lengths=[0])
    state, outs = case["state"].clone(), []
    for a, b in [(0, 67), (67, 147), (147, 148), (148, 149), (149, 150)]:
        part = {n: case[n][a:b] for n in ("q", "k", "v", "log_decay", "beta")}
        outs.append(nt.ninfer_gated_delta(**part, state=state, offsets=i32([0, b - a]) if b - a > 1 else None, lengths=i32([a]),
                                          norm_eps=1e-6, out_dtype=torch.float32))
    assert torch.allclose(torch.cat(outs), out, rtol=0, atol=2e-5 * out.abs().max().item())
    assert torch.allclose(state, whole, rtol=0, atol=2e-5 * whole.abs().max().item())


@pytest.mark.parametrize("dk", [96, 128, 256])
def test_gated_delta_waits_that_run_out(dk):
    """A bound of 0 makes every wait give up: the error word tells, no state or result of the call is stored, the next call is right."""
    rng = np.random.default_rng(14)
    case = delta_case(rng, 200, 2, 1, 2, dk, 64, "bf16")
    offsets, before, out = i32([0, 40, 200]), case["state"].clone(), torch.full((200, 2, 64), 5.0, device=DEV)
    assert nt.ninfer_device_errors() == 0
    nt.ninfer_set_wait_limit(0)
    try:
        nt.ninfer_gated_delta(**case, offsets=offsets, norm_eps=1e-6, out=out)
        torch.cuda.synchronize()
    finally:
        nt.ninfer_set_wait_limit(nt.WAIT_LIMIT_DEFAULT)
    assert nt.ninfer_device_errors() & 1 and nt.ninfer_device_errors() == 0
    assert torch.equal(case["state"], before) and (out == 5).all()
    run_delta(case, offsets=[0, 40, 200])


def test_gated_delta_extremes():
    """Decays that forget everything, states and values far apart in size, keys of zero, beta of zero and one."""
    rng = np.random.default_rng(10)
    for tokens, offsets in ((4, None), (90, [0, 1, 60, 90, 90])):
        case = delta_case(rng, tokens, 4, 1, 2, 128, 128, "bf16", 4)
        case["log_decay"] = case["log_decay"].clone()
        case["log_decay"][::5] = -200.0
        case["log_decay"][1::7] = 0.0
        case["beta"][::3] = 1.0
        case["beta"][1::4] = 0.0
        case["state"] *= f32(10.0 ** rng.integers(-12, 12, (4, 2, 1, 128)))
        case["k"][2 % tokens] = 0
        run_delta(case, offsets=offsets)


# ----------------------------------------------------------------- sample ---
def check_sample(x, random, **controls):
    """x (rows, vocab) on the GPU; controls as lists."""
    rows, vocab = x.shape
    logprobs = torch.full((rows,), 3.0, device=DEV)
    args = {n: (i32 if n == "top_k" else f32)(c) for n, c in controls.items()}
    tokens = nt.ninfer_sample(x, f32(random), logprobs=logprobs, **args)
    got, lp, wide = tokens.tolist(), f64(logprobs), f64(x)
    for b in range(rows):
        one = {n: float(np.float32(c[b])) if n != "top_k" else c[b] for n, c in controls.items()}
        want, p, near_ = ol.sample(wide[b], float(np.float32(random[b])), **one)
        if near_ < 2.0 ** -28:
            continue
        assert got[b] == want, (b, one, near_)
        assert lp[b] == p or abs(lp[b] - p) <= 2.0 ** -22 * (1 + abs(p)), (lp[b], p)
    return got


CONTROLS = [dict(), dict(temperature=0.7), dict(temperature=0.0), dict(top_k=5), dict(top_p=0.9), dict(min_p=0.05), dict(top_k=40, top_p=0.8),
            dict(top_k=100, min_p=0.02, temperature=1.5), dict(top_p=0.99, min_p=0.01, temperature=0.4), dict(top_k=1), dict(top_p=0.0),
            dict(min_p=1.0), dict(top_k=10 ** 9, top_p=1.0), dict(top_k=3, top_p=0.5, min_p=0.3, temperature=0.9)]
DEFAULT = dict(temperature=1.0, top_k=0, top_p=1.0, min_p=0.0)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [1, 2, 7, 33, 1000, 4099, 32003, 65536, 248320])
def test_sample(vocab, dtype):
    rng = np.random.default_rng(vocab)
    rows = 2 * len(CONTROLS)
    x = randn(rng, (rows, vocab + 5), dtype, 2.5)[:, :vocab] if vocab % 2 else randn(rng, (rows, vocab), dtype, 2.5)
    controls = {n: [{**DEFAULT, **CONTROLS[b % len(CONTROLS)]}[n] for b in range(rows)] for n in DEFAULT}
    random = rng.random(rows)
    random[0], random[1] = 0.0, 1 - 2.0 ** -24
    check_sample(x, random, **controls)


@pytest.mark.parametrize("rows,vocab,dtype", [(2, 1500001, "f32"), (1, 6000000, "bf16"), (40, 100003, "f16"), (200, 9001, "f32"), (330, 2049, "bf16")])
def test_sample_other_divisions(rows, vocab, dtype):
    """Rows too long for shared memory, rows of two to eight CTAs, of one."""
    g = torch.Generator("cuda").manual_seed(vocab)
    x = (torch.randn(rows, vocab, generator=g, device=DEV) * 2).to(TORCH[dtype])
    rng = np.random.default_rng(rows)
    pick = [CONTROLS[int(i)] for i in rng.integers(0, len(CONTROLS), rows)]
    pick[0] = dict(top_p=0.95)
    controls = {n: [{**DEFAULT, **c}[n] for c in pick] for n in DEFAULT}
    check_sample(x, rng.random(rows), **controls)


def test_sample_large_sets():
    """Nuclei and top-k of most of a row, borders inside thousands of equal logits."""
    rng = np.random.default_rng(21)
    x = randn(rng, (12, 60000), "f32", 0.3)
    x[6:] = (x[6:] * 4).round() / 4
    controls = dict(top_k=[0, 50000, 3000, 1500, 59999, 0, 0, 50000, 3000, 1500, 59999, 0],
                    top_p=[0.9, 1, 0.7, 1, 0.99, 0.9995, 0.9, 1, 0.7, 1, 0.99, 0.9995], temperature=[1, 2, 1, 1, 0.5, 3] * 2)
    for seed in range(3):
        check_sample(x, np.random.default_rng(seed).random(12), **controls)
    check_sample(x, rng.random(12), min_p=[0.2] * 12)


def test_sample_one_row_without_controls():
    rng = np.random.default_rng(4)
    x = randn(rng, (1, 248320), "f32", 3)
    for r in (0.0, 0.123, 0.5, 0.99999):
        check_sample(x, [r])
        check_sample(x, [r], top_p=[0.95])


def test_sample_ties_are_kept_in_order():
    """Equal logits at every border: the lower places stay."""
    x = torch.zeros(6, 5000, device=DEV)
    x[:, 1000:2000] = 1.0
    x[:, 1500] = -0.0
    x[5] = -0.0
    got = check_sample(x, [0.999999, 0.999999, 0.5, 0.0, 0.999, 0.25], top_k=[10, 1009, 0, 0, 0, 0], top_p=[1, 1, 0.25, 0.25, 1, 0.5],
                       min_p=[0, 0, 0, 0, 1.0, 0])
    # row 1 keeps the 999 ones and the first ten zeros; the last of them in the row's order is a one
    assert got[0] == 1009 and got[1] == 1999 and got[3] == 1000 and 0 <= got[5] < 2500


def test_sample_masks_infinities_and_nan():
    x = torch.full((8, 3001), -float("inf"), device=DEV)
    x[1, 2999] = -1e30
    x[2, 5:8] = float("inf")
    x[3] = float("nan")
    x[4, 100:200] = torch.finfo(torch.float32).min
    x[5, ::2] = 1.0
    x[5, 1::2] = float("nan")
    x[6, 17], x[6, 18] = 3e38, -3e38
    x[7, 3000] = 0.0
    r = [0.5] * 8
    got = check_sample(x, r)
    assert got[0] == -1 and got[1] == 2999 and got[2] == 6 and got[3] == -1 and got[4] == 150 and got[5] % 2 == 0 and got[6] == 17 and got[7] == 3000
    assert check_sample(x, r, top_k=[4] * 8, top_p=[0.9] * 8, min_p=[0.1] * 8)[2] == 6
    assert check_sample(x, r, temperature=[0.0] * 8) == [-1, 2999, 5, -1, 100, 0, 17, 3000]


@pytest.mark.parametrize("temperature", [1e-30, 1e-6, 1e-3, 30.0, 1e6, float("inf"), float("nan"), -1.0])
def test_sample_temperatures(temperature):
    rng = np.random.default_rng(5)
    x = randn(rng, (4, 2000), "f32", 4)
    check_sample(x, [0.1, 0.5, 0.9, 0.3], temperature=[temperature] * 4, top_p=[1.0, 0.7, 1.0, 0.2], top_k=[0, 0, 7, 0])


def test_sample_controls_out_of_range():
    rng = np.random.default_rng(6)
    x = randn(rng, (7, 999), "f32", 2)
    nan = float("nan")
    got = check_sample(x, [0.3] * 7, top_p=[nan, -1.0, 2.0, 1.0, 1.0, 1.0, 1.0], min_p=[0, 0, 0, nan, 7.0, -2.0, 0], top_k=[0, 0, 0, 0, 0, -4, 2 ** 31 - 1])
    top = x.argmax(1).tolist()
    assert got[1] == top[1] and got[4] == top[4]
    lp = torch.empty(2, device=DEV)
    edge = nt.ninfer_sample(x[:2], f32([2.0, nan]), logprobs=lp)       # cut to 1 and 0: the last and the first token
    assert edge.tolist() == [998, 0]


def test_sample_equal_rows_give_equal_tokens():
    """However a row is divided and wherever it lies, its sums are the same whole numbers."""
    rng = np.random.default_rng(11)
    row = randn(rng, (1, 50021), "f32", 2)
    random, n = rng.random(50), 50
    x = row.expand(n, -1).contiguous()
    batch = nt.ninfer_sample(x, f32(random), top_p=f32([0.97] * n)).tolist()
    ones = [int(nt.ninfer_sample(row, f32([r]), top_p=f32([0.97]))) for r in random]
    assert batch == ones


# ----------------------------------------------------- streams and graphs ---
def test_calls_on_a_stream_and_in_a_graph():
    """The operators in a captured graph, replayed on new inputs, give what the calls give."""
    rng = np.random.default_rng(12)
    x, w = randn(rng, (5, 512)), randn(rng, (512,))
    case = delta_case(rng, 5, 5, 1, 2, 64, 128, "f32")
    q, freq = randn(rng, (5, 4, 64)), torch.from_numpy(nt.ninfer_rotary_frequencies(64)[0]).to(DEV)
    logits, random = randn(rng, (5, 3000)), f32(rng.random(5))
    bufs = dict(norm=torch.empty_like(x), q=torch.empty_like(q), out=torch.empty(5, 2, 128, device=DEV), token=torch.empty(5, dtype=torch.int32, device=DEV))
    positions = i32(np.arange(5))

    def step():
        nt.ninfer_norm(x, w, out=bufs["norm"])
        nt.ninfer_rotary(q, None, positions, freq, q_out=bufs["q"])
        nt.ninfer_gated_delta(**case, norm_eps=1e-6, out=bufs["out"])
        nt.ninfer_sample(logits, random, top_p=f_p, out=bufs["token"])
    f_p = f32([0.9] * 5)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    kept = case["state"].clone()
    with torch.cuda.stream(stream):
        step()
    stream.synchronize()
    case["state"].copy_(kept)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for seed in range(3):
        g = torch.Generator("cuda").manual_seed(seed)
        for t in (x, q, logits, case["q"], case["k"], case["v"]):
            t.copy_(torch.randn(t.shape, generator=g, device=DEV))
        positions.add_(1000)
        case["state"].copy_(kept)
        step()
        torch.cuda.synchronize()
        eager = [t.clone() for t in (*bufs.values(), case["state"])]
        case["state"].copy_(kept)
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(eager, (*bufs.values(), case["state"])):
            assert torch.equal(a, b)


def test_binding_refusals():
    x = torch.zeros(3, 64, device=DEV)
    with pytest.raises(ValueError):
        nt.ninfer_norm(x.cpu())
    with pytest.raises(ValueError):
        nt.ninfer_norm(x, torch.ones(63, device=DEV))
    with pytest.raises(ValueError):
        nt.ninfer_norm(x, residual=x, sum=torch.empty(3, 64, dtype=torch.bfloat16, device=DEV))
    with pytest.raises(ValueError):
        nt.ninfer_norm(x.t())
    with pytest.raises(ValueError):
        nt.ninfer_norm(x, gate=x[:2])
    q, freq, pos = torch.zeros(3, 2, 64, device=DEV), torch.zeros(32, dtype=torch.int64, device=DEV), torch.zeros(3, dtype=torch.int32, device=DEV)
    for bad in (dict(k=q[:2]), dict(k=q.bfloat16()), dict(k=None, k_out=q), dict(positions=pos.long()), dict(positions=pos[:2]),
                dict(q_weight=torch.ones(32, device=DEV)), dict(q_out=q[:, :1]), dict(frequencies=freq.int())):
        with pytest.raises(ValueError):
            nt.ninfer_rotary(**{**dict(q=q, k=None, positions=pos, frequencies=freq), **bad})
    case = delta_case(np.random.default_rng(0), 3, 3, 1, 2, 64, 64, "f32")
    for bad in (dict(k=case["k"][:, :, :32]), dict(v=case["v"].bfloat16()), dict(beta=case["beta"].half()), dict(beta=case["beta"][:, :1]),
                dict(state=case["state"][:, :1]), dict(state=case["state"].transpose(2, 3)), dict(offsets=pos.long()), dict(lengths=pos[:2]),
                dict(out=torch.empty(3, 2, 32, device=DEV)), dict(slots=torch.zeros(4, dtype=torch.int64, device=DEV))):
        with pytest.raises(ValueError):
            nt.ninfer_gated_delta(**{**case, **bad})
    with pytest.raises(nt.NinferError):
        nt.ninfer_gated_delta(**case, slots=torch.zeros(2, dtype=torch.int32, device=DEV))
    r = torch.zeros(3, device=DEV)
    for bad in (dict(random=r[:2]), dict(top_k=r), dict(top_p=r.double()), dict(out=torch.empty(3, dtype=torch.int64, device=DEV)), dict(logprobs=r.half())):
        with pytest.raises(ValueError):
            nt.ninfer_sample(**{**dict(logits=x, random=r), **bad})
