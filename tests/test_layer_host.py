"""Operators of a layer's step, the part that needs no GPU: hand-worked values of
the oracle, the table of rotary frequencies, and the refusals, which come back
before any device work (fake aligned addresses stand in for device buffers)."""
import math

import numpy as np
import pytest

import bit_gemv_gb300 as nt
from oracle import layer as ol

INVALID, SHAPE, SIZE, ALIGN, OVERFLOW = 1, 3, 4, 5, 8
FAKE = 1 << 20
lib = nt._lib


# ----------------------------------------------------------------- oracle ---
def test_oracle_norm_by_hand():
    # (1, 7) + (2, -3) = (3, 4): mean square 12.5
    s, y = ol.norm([[1.0, 7.0]], np.array([[2.0, -3.0]]), None, [0.5, 1.0], None, 0.0, 0.5)
    assert s.tolist() == [[3, 4]] and np.allclose(y, [[3 / math.sqrt(12.5), 6 / math.sqrt(12.5)]])
    # two groups; a gate of ln 3 is ln 3 * 3 / 4
    _, y = ol.norm([[2.0, 0.0]], None, np.array([[math.log(3), 1.0]]), None, 1, 0.0)
    assert np.allclose(y[0, 0], math.log(3) * 0.75) and np.isnan(ol.norm([[0.0]], None, None, None, 1, 0.0)[1][0, 0])


def test_oracle_rotary_by_hand():
    quarter = 2 ** 62
    x = np.arange(1.0, 5.0).reshape(1, 1, 4)
    assert np.allclose(ol.rotary(x, [1], [quarter, 0]), [[[-3, 2, 1, 4]]])
    assert np.allclose(ol.rotary(x, [3], [quarter, 0], 2.0, True), [[[4, -2, 6, 8]]])
    assert np.allclose(ol.rotary(x, [2 ** 31 - 1], [quarter]), [[[2, -1, 3, 4]]])        # 3 quarters once whole turns are gone


def test_oracle_gated_delta_by_hand():
    # one column: S = (2, 0) -> halved (1, 0); k = (1, 0), v = 3, beta = 1/2: u = 1, S = (2, 0); q = (1, 1): 2
    q, k = np.array([[[1.0, 1.0]]]), np.array([[[1.0, 0.0]]])
    out, s, _, _ = ol.gated_delta(q, k, np.array([[[3.0]]]), np.array([[math.log(0.5)]]), np.array([[0.5]]),
                                  np.array([[[[2.0], [0.0]]]]), [0, 1], [0])
    assert np.allclose(out, 2) and np.allclose(s.ravel(), [2, 0])
    # beta = 1 and a key of norm 1: the state answers with the value just learnt
    out, s, _, _ = ol.gated_delta(k, k, np.array([[[7.0]]]), np.zeros((1, 1)), np.ones((1, 1)), np.array([[[[2.0], [5.0]]]]), [0, 1], [0], [0])
    assert np.allclose(out, 7) and np.allclose(s.ravel(), [7, 0])


def test_oracle_sample_by_hand():
    x = np.log([0.1, 0.4, 0.3, 0.2])
    assert [ol.sample(x, r)[0] for r in (0.0, 0.09, 0.11, 0.49, 0.51, 0.79, 0.81, 1.0)] == [0, 0, 1, 1, 2, 2, 3, 3]
    assert [ol.sample(x, r, top_k=2)[0] for r in (0.0, 0.56, 0.58)] == [1, 1, 2]
    assert [ol.sample(x, r, top_p=0.65)[0] for r in (0.0, 0.56, 0.58)] == [1, 1, 2]         # 0.4 + 0.3
    assert [ol.sample(x, r, min_p=0.6)[0] for r in (0.0, 0.58)] == [1, 2]
    assert ol.sample(x, 0.9, temperature=0)[:2] == (1, 0.0) and ol.sample(x, 0.9, top_p=0)[0] == 1
    assert np.isclose(ol.sample(x, 0.58, top_k=2)[1], math.log(3 / 7))
    assert ol.sample([-np.inf, np.nan], 0.5)[0] == -1 and ol.sample([1.0, np.inf, np.inf], 0.6)[0] == 2


# ------------------------------------------------------------ frequencies ---
@pytest.mark.parametrize("scaling,args", [("none", {}), ("linear", dict(factor=4.0)),
                                          ("dimensions", dict(factor=8.0, context=32768.0)),
                                          ("dimensions", dict(factor=40.0, context=4096.0, slow=0.5, fast=64.0)),
                                          ("turns", dict(factor=8.0, context=8192.0, slow=1.0, fast=4.0))])
@pytest.mark.parametrize("dim,base", [(2, 10000.0), (64, 1e6), (128, 500000.0), (256, 10000.0), (20, 1.5)])
def test_rotary_frequencies(scaling, args, dim, base):
    got, magnitude = nt.ninfer_rotary_frequencies(dim, base, scaling, **args)
    want, m = ol.rotary_frequencies(dim, base, scaling, **args)
    assert got.dtype == np.int64 and got.shape == (dim // 2,)
    # 53-bit arithmetic of a few steps, then whole 2^-64 turns
    turns = got.view(np.uint64).astype(np.float64) / 2.0 ** 64
    assert np.all(np.abs(turns - want / (2 * np.pi)) <= 2.0 ** -64 + 2.0 ** -48 * turns)
    assert magnitude == np.float32(m)


def test_rotary_frequencies_refusals():
    bad = [dict(rotary_dim=0), dict(rotary_dim=3), dict(rotary_dim=258), dict(base=1.0), dict(base=float("nan")),
           dict(scaling="linear", factor=0.5), dict(scaling="dimensions", factor=2.0, context=0.0),
           dict(scaling="turns", factor=2.0, context=10.0, slow=2.0, fast=2.0), dict(scaling="turns", factor=float("inf"), context=10.0)]
    for b in bad:
        with pytest.raises(nt.NinferError):
            nt.ninfer_rotary_frequencies(**{**dict(rotary_dim=64), **b})
    with pytest.raises(ValueError):
        nt.ninfer_rotary_frequencies(64, scaling="other")
    assert lib.ninfer_rotary_frequencies(64, 1e4, 9, 1.0, 1.0, 1.0, 2.0, np.zeros(32, np.uint64).ctypes.data, nt.C.byref(nt.C.c_float())) == INVALID
    assert lib.ninfer_rotary_frequencies(64, 1e4, 0, 1.0, 1.0, 1.0, 2.0, None, nt.C.byref(nt.C.c_float())) == INVALID


# --------------------------------------------------------------- refusals ---
NORM = ["x", "residual", "gate", "weight", "sum", "out", "rows", "cols", "group", "x_stride", "residual_stride", "gate_stride",
        "sum_stride", "out_stride", "eps", "weight_offset", "x_dtype", "residual_dtype", "gate_dtype", "weight_dtype", "out_dtype", "reserved"]


def norm(**kw):
    a = dict(zip(NORM, [FAKE * (i + 1) for i in range(6)] + [4, 64, 64] + [64] * 5 + [1e-6, 0.0] + [nt.BF16] * 5 + [0]))
    a.update(kw)
    return lib.ninfer_norm(nt._NORM.pack(*[a[n] for n in NORM]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(x=0), INVALID), (dict(out=0), INVALID), (dict(residual=0), INVALID), (dict(reserved=1), INVALID), (dict(eps=-1.0), INVALID),
    (dict(eps=float("nan")), INVALID), (dict(eps=float("inf")), INVALID), (dict(weight_offset=float("inf")), INVALID),
    (dict(rows=0), SHAPE), (dict(cols=0), SHAPE), (dict(group=0), SHAPE), (dict(group=48), SHAPE), (dict(group=128), SHAPE),
    (dict(cols=2 ** 31, group=2 ** 31, x_stride=2 ** 31), SHAPE), (dict(x_stride=63), SHAPE), (dict(sum_stride=8), SHAPE),
    (dict(gate_stride=0), SHAPE), (dict(x_dtype=3), INVALID), (dict(out_dtype=-1), INVALID), (dict(weight_dtype=9), INVALID),
    (dict(x=FAKE + 1), ALIGN), (dict(weight=FAKE + 2, weight_dtype=nt.F32), ALIGN), (dict(out_stride=2 ** 40), OVERFLOW),
    (dict(rows=2 ** 31), OVERFLOW), (dict(rows=2 ** 26, group=1), OVERFLOW), (dict(rows=2 ** 63, group=1), OVERFLOW),
    # in place with another stride or type, outputs over each other or over other inputs
    (dict(out=FAKE, out_stride=72), INVALID), (dict(out=FAKE, out_dtype=nt.F16), INVALID), (dict(out=FAKE * 3, gate_stride=72), INVALID),
    (dict(out=FAKE * 3, gate_dtype=nt.F16), INVALID), (dict(sum=FAKE * 2, sum_stride=72), INVALID), (dict(out=FAKE * 2), INVALID),
    (dict(out=FAKE * 5), INVALID), (dict(sum=FAKE), INVALID), (dict(sum=FAKE * 3), INVALID)])
def test_norm_refusals(kw, status):
    assert norm(**kw) == status
    assert lib.ninfer_norm(None, None) == INVALID


ROTARY = ["q", "k", "q_weight", "k_weight", "q_out", "k_out", "positions", "frequencies", "tokens", "q_heads", "kv_heads", "head_dim",
          "rotary_dim", "q_token", "q_head", "k_token", "k_head", "q_out_token", "q_out_head", "k_out_token", "k_out_head", "magnitude",
          "eps", "weight_offset", "dtype", "weight_dtype", "interleaved"]


def rotary(**kw):
    a = dict(zip(ROTARY, [FAKE, 2 * FAKE, FAKE, FAKE, FAKE, 2 * FAKE, FAKE, FAKE] + [3, 4, 2, 64, 32] + [256, 64, 128, 64] * 2 + [1.0, 1e-6, 0.0, nt.BF16, nt.F32, 0]))
    a.update(kw)
    return lib.ninfer_rotary(nt._ROTARY.pack(*[a[n] for n in ROTARY]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(q=0), INVALID), (dict(q_out=0), INVALID), (dict(k_out=0), INVALID), (dict(k=0), INVALID), (dict(positions=0), INVALID),
    (dict(frequencies=0), INVALID), (dict(dtype=3), INVALID), (dict(weight_dtype=4), INVALID), (dict(magnitude=float("nan")), INVALID),
    (dict(eps=-1e-6), INVALID), (dict(weight_offset=float("inf")), INVALID), (dict(tokens=0), SHAPE), (dict(tokens=2 ** 31), SHAPE),
    (dict(q_heads=0), SHAPE), (dict(kv_heads=0), SHAPE), (dict(q_heads=65536), SHAPE), (dict(head_dim=60), SHAPE), (dict(head_dim=264), SHAPE),
    (dict(rotary_dim=0), SHAPE), (dict(rotary_dim=31), SHAPE), (dict(rotary_dim=66), SHAPE), (dict(q=FAKE + 8), ALIGN),
    (dict(k_out=FAKE + 2), ALIGN), (dict(q_token=260), ALIGN), (dict(k_out_head=65), ALIGN), (dict(positions=FAKE + 2), ALIGN),
    (dict(frequencies=FAKE + 4), ALIGN), (dict(q_weight=FAKE + 4), ALIGN), (dict(k_token=2 ** 40), OVERFLOW),
    (dict(q_out_token=512), INVALID), (dict(k_out_head=128), INVALID), (dict(q_out=2 * FAKE), INVALID), (dict(k_out=FAKE), INVALID)])
def test_rotary_refusals(kw, status):
    assert rotary(**kw) == status
    assert lib.ninfer_rotary(None, None) == INVALID


DELTA = ["q", "k", "v", "log_decay", "beta", "state", "state_slots", "offsets", "lengths", "out", "status", "tokens", "requests", "slots",
         "k_heads", "v_heads", "k_dim", "v_dim", "q_token", "q_head", "k_token", "k_head", "v_token", "v_head", "decay_stride", "beta_stride",
         "slot_stride", "scale", "norm_eps", "dtype", "out_dtype"]


def delta(workspace=FAKE, bytes_=2 ** 40, **kw):
    a = dict(zip(DELTA, [FAKE] * 11 + [9, 3, 5, 2, 4, 64, 32] + [128, 64, 128, 64, 128, 32] + [4, 4, 8192] + [0.125, 1e-6, nt.BF16, nt.BF16]))
    a.update(kw)
    return lib.ninfer_gated_delta(nt._DELTA.pack(*[a[n] for n in DELTA]), workspace, bytes_, None)


@pytest.mark.parametrize("kw,status", [
    *[({n: 0}, INVALID) for n in ("q", "k", "v", "log_decay", "beta", "state", "out")], (dict(dtype=3), INVALID), (dict(out_dtype=5), INVALID),
    (dict(scale=float("nan")), INVALID), (dict(norm_eps=float("inf")), INVALID), (dict(tokens=0), SHAPE), (dict(tokens=2 ** 31), SHAPE),
    (dict(requests=0), SHAPE), (dict(k_heads=0), SHAPE), (dict(v_heads=0), SHAPE), (dict(v_heads=5), SHAPE), (dict(v_heads=65536), SHAPE),
    (dict(k_dim=60), SHAPE), (dict(k_dim=264), SHAPE), (dict(v_dim=0), SHAPE), (dict(v_dim=4), SHAPE), (dict(offsets=0), SHAPE),
    (dict(slots=0), SHAPE), (dict(slots=2, state_slots=0), SHAPE), (dict(slot_stride=8188), SHAPE), (dict(decay_stride=3), SHAPE),
    (dict(beta_stride=0), SHAPE), (dict(q=FAKE + 8), ALIGN), (dict(q_token=132), ALIGN), (dict(v_head=33), ALIGN), (dict(k_token=2 ** 40), OVERFLOW),
    (dict(slot_stride=2 ** 40), OVERFLOW), (dict(slot_stride=8194), ALIGN), (dict(state=FAKE + 4), ALIGN), (dict(out=FAKE + 8), ALIGN),
    (dict(offsets=FAKE + 1), ALIGN), (dict(log_decay=FAKE + 2), ALIGN), (dict(status=FAKE + 2), ALIGN),
    (dict(requests=2 ** 31 - 1, v_heads=4096, k_heads=1, slots=2 ** 31 - 1, slot_stride=2 ** 32, decay_stride=4096, beta_stride=4096, bytes_=2 ** 63), OVERFLOW)])
def test_gated_delta_refusals(kw, status):
    assert delta(**kw) == status
    assert lib.ninfer_gated_delta(None, None, 0, None) == INVALID


def test_gated_delta_workspace_refusals():
    assert lib.ninfer_gated_delta_workspace(9, 3, 2, 4, 64, 32, None) == INVALID
    for bad in ((0, 3, 2, 4, 64, 32), (9, 0, 2, 4, 64, 32), (9, 3, 0, 4, 64, 32), (9, 3, 2, 5, 64, 32), (9, 3, 2, 4, 63, 32), (9, 3, 2, 4, 64, 512)):
        with pytest.raises(nt.NinferError):
            nt.ninfer_gated_delta_workspace(*bad)
    need = nt.ninfer_gated_delta_workspace(900, 3, 2, 4, 128, 128)
    if need:
        args = dict(tokens=900, k_dim=128, v_dim=128, slot_stride=65536, q_token=256, q_head=128, k_token=256, k_head=128, v_token=512, v_head=128)
        assert delta(None, 0, **args) == INVALID
        assert delta(FAKE, need - 1, **args) == SIZE
        assert delta(FAKE + 128, need, **args) == ALIGN


SAMPLE = ["logits", "temperature", "top_p", "min_p", "top_k", "random", "tokens", "logprobs", "rows", "vocab", "stride", "dtype", "reserved"]


def sample(**kw):
    a = dict(zip(SAMPLE, [FAKE] * 8 + [3, 100, 100, nt.F32, 0]))
    a.update(kw)
    return lib.ninfer_sample(nt._SAMPLE.pack(*[a[n] for n in SAMPLE]), None)


@pytest.mark.parametrize("kw,status", [
    (dict(logits=0), INVALID), (dict(random=0), INVALID), (dict(tokens=0), INVALID), (dict(dtype=3), INVALID), (dict(reserved=2), INVALID),
    (dict(rows=0), SHAPE), (dict(vocab=0), SHAPE), (dict(vocab=2 ** 30 + 1), SHAPE), (dict(stride=99), SHAPE), (dict(rows=2 ** 31), OVERFLOW),
    (dict(stride=2 ** 40), OVERFLOW), (dict(logits=FAKE + 2), ALIGN), (dict(top_k=FAKE + 2), ALIGN), (dict(logprobs=FAKE + 1), ALIGN)])
def test_sample_refusals(kw, status):
    assert sample(**kw) == status
    assert lib.ninfer_sample(None, None) == INVALID
