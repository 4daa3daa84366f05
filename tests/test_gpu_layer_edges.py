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
