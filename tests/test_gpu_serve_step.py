"""The loop of examples/serve_step.py: prompts at once and single tokens through
norms, rotary positions, gated delta, attention and sampling as a program uses
them, each operator of every step held to its fp64 definition on what it got."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import bit_gemv_gb300 as nt
from oracle import layer as ol
from test_gpu_layer import f64, near

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
U = 2.0 ** -24


@pytest.fixture(scope="module")
def ex():
    spec = importlib.util.spec_from_file_location("serve_step_example", os.path.join(ROOT, "examples", "serve_step.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


PROMPTS = [list(range(7, 60)), [1], [4000, 17, 17, 3] * 10]


def test_steps_against_the_definitions(ex):
    server = ex.Server(ex.Model(), PROMPTS, longest=64, page=16, watch=True)
    states = None
    for step in range(5):
        logits = server.step()
        assert torch.isfinite(logits).all()
        deltas = 0
        for kind, got, gave, more in server.seen[step]:
            if kind == "norm":
                x, residual, gate, weight, group = (f64(t) if torch.is_tensor(t) else t for t in got)
                s, want = ol.norm(x, residual, gate, weight, group, ex.EPS)
                near(f64(gave[1]), want, 40 * U * np.abs(want), "bf16")
                if gave[0] is not None:
                    near(f64(gave[0]), s, U * np.abs(s), "f32")
            elif kind == "rotary":
                turns = server.model.frequencies.cpu().numpy().view(np.uint64)
                for x, y, w in zip(got, gave, more[1:]):
                    want = ol.rotary(f64(x), more[0].tolist(), turns, server.model.magnitude, False, f64(w), ex.EPS)
                    size = np.linalg.norm(want, axis=-1, keepdims=True)         # no pair is larger
                    near(f64(y), want, 2.0 ** -19 * size, "bf16")
            elif kind == "delta":
                offsets = np.concatenate([[0], np.cumsum(more)])
                before = np.zeros((3, ex.V_HEADS, ex.DELTA_DIM, ex.DELTA_DIM)) if states is None else states[deltas]
                want, state, out_bound, bound = ol.gated_delta(*map(f64, got), before, offsets, range(3), None, ex.DELTA_DIM ** -0.5, ex.EPS,
                                                               2.0 ** -23, 2.0 ** -39 if step == 0 else 0.0)
                near(f64(gave), want, out_bound, "bf16")
                held = [h for h, k in zip(server.held, ex.LAYERS) if k == "delta"][deltas]
                near(f64(held), state, bound, "f32")
                deltas += 1
            else:
                for b in range(3):
                    token, _, border = ol.sample(f64(got[0])[b], float(got[1][b]), 0.0 if b == 0 else float(np.float32(0.8)), 0, float(np.float32(0.95)))
                    assert border < 2.0 ** -24 or int(gave[b]) == token
        states = [f64(h) for h, k in zip(server.held, ex.LAYERS) if k == "delta"]
        assert server.lengths.tolist() == [len(p) + step for p in PROMPTS]
    for r, p in enumerate(PROMPTS):
        assert server.history[r, :len(p)].tolist() == p
    assert nt.ninfer_device_errors() == 0


def test_runs_repeat_and_pages_do_not_matter(ex):
    """The same answers, bit for bit, from another run and from other pages."""
    model, runs = ex.Model(), []
    for page, seed in ((16, 1), (16, 1), (7, 1), (64, 1)):
        server = ex.Server(model, PROMPTS, longest=80, page=page, seed=seed)
        logits = torch.stack([server.step() for _ in range(12)])
        runs.append((logits, server.history.clone()))
        assert logits[:, 0].argmax(-1).tolist() == server.history[0, len(PROMPTS[0]):len(PROMPTS[0]) + 12].tolist()
    for logits, history in runs[1:]:
        assert torch.equal(logits, runs[0][0]) and torch.equal(history, runs[0][1])
