"""Operators of a layer's step on the GPU where they went, or could go, wrong; against their fp64 definitions and against
themselves. Bounds as in test_gpu_layer.py unless derived here."""
import numpy as np
import pytest
import torch

import bit_gemv_gb300 as nt
from oracle import layer as ol
from test_gpu_layer import DEV, HALF, TORCH, delta_case, f32, f64, i32, near, randn, run_delta

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
