"""The decode loop of examples/decode_step.py: its operators together, as a
program uses them, checked step by step against the fp64 definitions."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import bit_gemv_gb300 as nt
from oracle import decode as od

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("decode_step_example", os.path.join(ROOT, "examples", "decode_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


PROMPTS = [[5, 9, 2], [1], [4000, 17, 17, 17, 3, 2, 1]]


def test_steps_against_the_definitions(ex):
    """Every layer's attention of every step against fp64 attention over the keys and values that the
    projections gave so far; the allowed tokens and the answers of the loop."""
    model = ex.Model()
    d = ex.Decoder(model, PROMPTS, longest=40, page=16)
    seen = [[] for _ in model.layers]
    scale = ex.HEAD_DIM ** -0.5
    for i in range(36):
        logits = d.step()
        for kept, (qkv, a) in zip(seen, d.attended):
            kept.append(f64(qkv))
            k = np.stack([x[:, ex.HEADS:ex.HEADS + ex.KV_HEADS] for x in kept], 1)      # request, token, head, element
            v = np.stack([x[:, ex.HEADS + ex.KV_HEADS:] for x in kept], 1)
            want, _, mag, big = od.kv_attention(kept[-1][:, :ex.HEADS], k, v, np.arange(3)[:, None], [i + 1] * 3, scale)
            bound = (2 * big[..., None] + 1) * 2.0 ** -15 * mag + 2.0 ** -8 * np.abs(want)
            assert (np.abs(f64(a) - want) <= bound).all(), i
        assert (logits[0, 1::2] == -float("inf")).all() and torch.isfinite(logits[1:]).all()
        assert d.lengths.tolist() == [i + 1] * 3
    for r, p in enumerate(PROMPTS):
        assert d.history[r, :len(p)].tolist() == p
    assert (d.history[0, 3:37] % 2 == 0).all()
    used = d.block_table[d.block_table >= 0].tolist()
    assert len(used) == 9 and len(set(used)) == 9
    assert nt.ninfer_device_errors() == 0


def test_pages_do_not_change_the_answers(ex):
    """Other page sizes, and other pages of the pool, give the same logits bit for bit."""
    model = ex.Model()
    runs = []
    for page, seed in ((16, 1), (16, 2), (7, 3), (1, 4), (64, 5)):
        d = ex.Decoder(model, PROMPTS, longest=40, page=page, seed=seed)
        runs.append(torch.stack([d.step() for _ in range(30)]))
    for r in runs[1:]:
        assert torch.equal(r, runs[0])


def test_eight_bit_cache(ex):
    """The loop on an 8-bit cache: the first step attends to one key, so only its value's rounding shows."""
    model = ex.Model()
    a = ex.Decoder(model, PROMPTS, longest=8, cache_dtype=torch.float8_e4m3fn)
    a.step()
    qkv, out = a.attended[0]
    v = od.round_to(f64(qkv[:, ex.HEADS + ex.KV_HEADS:]), "e4m3", True)
    want = np.repeat(v, ex.HEADS // ex.KV_HEADS, axis=1)
    assert np.array_equal(f64(out), want)
