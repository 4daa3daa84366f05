"""Decode-step operators on the GPU where results are easily lost: NaN and infinities on
every path of the attention, and sums and roundings held to the arithmetic that the header states.

The attention has three paths, chosen from the block table's width: a CTA a row, a cluster
of CTAs a row, and the division of all keys with a second kernel. Only the last one writes to
its workspace, which is how a test sees that it reached the path that it is about."""
import copy

import numpy as np
import pytest
import torch

import bit_gemv_gb300 as nt
from oracle import decode as od

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


def attend(q, k, v, table, lengths, width, **kw):
    """Attention under a block table of `width` pages a row; returns out, lse and whether the keys were divided."""
    wide = np.full((len(lengths), width), -1, np.int64)
    wide[:, :np.shape(table)[1]] = table
    cache = nt.KvCache(k, v)
    ws = torch.full((nt.ninfer_kv_attention_workspace(cache, *q.shape[:2]),), 0xa5, dtype=torch.uint8, device=DEV)
    lse = torch.zeros(q.shape[:2], device=DEV)
    out = nt.ninfer_kv_attention(q, cache, i32(wide), i32(lengths), scale=q.shape[2] ** -0.5, lse=lse, workspace=ws, **kw)
    return out, lse, bool((ws != 0xa5).any())


# 200 keys in 13 pages of 16; tables this wide lead to one CTA, clusters of 2, 4 and 8, and the division
# (rows of 128 elements in 16 bits are 32 keys a unit: 7, 15, 30, 60 and 200 units)
WIDTHS = {13: False, 30: False, 60: False, 120: False, 400: True}


@pytest.mark.parametrize("width", WIDTHS)
@pytest.mark.parametrize("group", [1, 8, 16])
@pytest.mark.parametrize("what", ["query", "one head's query", "keys", "last key", "values", "-inf keys", "-inf keys of infinite values"])
def test_attention_nan_and_infinity_on_every_path(what, group, width):
    rng = np.random.default_rng(group)
    q, k, v = (torch.from_numpy(rng.standard_normal(s).astype(np.float32)).to(DEV).bfloat16()
               for s in ((1, 2 * group, 128), (13, 16, 2, 128), (13, 16, 2, 128)))
    # what is spoilt lies in key head 0 (query heads below `group`); key head 1 stays clean
    if what == "query":
        q[0, :group] = float("nan")
    elif what == "one head's query":
        q[0, 0, 5] = float("nan")
    elif what == "keys":
        k[4:6, :, 0] = float("nan")            # one unit of 32 keys, all that a CTA of eight has
    elif what == "last key":
        k[12, 7, 0, 127] = float("nan")
    elif what == "values":
        v[4:6, :, 0, 3] = float("nan")
    else:
        q[0, :group, 0], k[4:6, :, 0, 0] = 1.0, -float("inf")
        if "values" in what:
            v[4, 0, 0, 9] = float("inf")
    out, lse, divided = attend(q, k, v, [list(range(13))], [200], width)
    assert divided == WIDTHS[width]
    with np.errstate(invalid="ignore"):
        want, wlse, _, _ = od.kv_attention(f64(q), f64(k), f64(v), np.arange(13)[None], [200], 128 ** -0.5)
    if "values" in what and "inf" in what:
        want[0, :group, 9] = np.nan            # a weight of 0 times an infinite value
    got, glse = f64(out), f64(lse)
    assert np.array_equal(np.isnan(got), np.isnan(want)) and np.array_equal(np.isnan(glse), np.isnan(wlse))
    fine, lfine = np.isfinite(want), np.isfinite(wlse)
    # scores of deviation one, averages of standard normal values: 2^-6 is eight steps of a bfloat16 result near one
    assert np.abs(got - want)[fine].max(initial=0) < 2.0 ** -6 and np.abs(glse - wlse)[lfine].max(initial=0) < 2.0 ** -10


@pytest.mark.parametrize("width", WIDTHS)
def test_attention_rows_of_minus_infinity_on_every_path(width):
    q = torch.ones(1, 8, 128, dtype=torch.bfloat16, device=DEV)
    k, v = torch.zeros(13, 16, 1, 128, dtype=torch.bfloat16, device=DEV), torch.ones(13, 16, 1, 128, dtype=torch.bfloat16, device=DEV)
    k[..., 0] = -float("inf")
    out, lse, _ = attend(q, k, v, [list(range(13))], [200], width)
    assert (out == 0).all() and (lse == -float("inf")).all()


@pytest.mark.parametrize("cache", ["f16", "e4m3", "bf16"])
@pytest.mark.parametrize("q_dtype,out", [("f32", "f32"), ("bf16", "bf16"), ("f32", "bf16")])
@pytest.mark.parametrize("factor", [1.0, 1e30, 1e-30])
def test_attention_query_elements_far_below_the_largest(cache, q_dtype, out, factor):
    """A query's largest element meets keys of zero, so that elements 2^-20 of it decide.

    A score may be 2^-15 of sum |q k| scale off, a weight by twice that and by its own rounding (2^-12 at most), and the
    result's format adds half a step."""
    rng = np.random.default_rng(11)
    q = torch.from_numpy(rng.standard_normal((1, 4, 64)).astype(np.float32)).to(DEV) * 2
    q[:, :, 7] = torch.tensor([2.0 ** 20, -1.9 * 2.0 ** 20, 2.0 ** 20, 1.0], device=DEV)
    q = (q * factor).to(TORCH[q_dtype])
    k, v = (torch.from_numpy(rng.standard_normal((4, 16, 1, 64)).astype(np.float32)).to(DEV).to(TORCH[cache]) for _ in range(2))
    (k.view(torch.uint8) if cache == "e4m3" else k)[..., 7] = 0
    y = nt.ninfer_kv_attention(q, nt.KvCache(k, v), i32([[0, 1, 2, 3]]), i32([61]), scale=0.125 / factor, out_dtype=TORCH[out])
    want, _, mag, big = od.kv_attention(f64(q), f64(k), f64(v), np.arange(4)[None], [61], np.float32(0.125 / factor).astype(np.float64))
    bound = (2 * big[..., None] * 2.0 ** -15 + 2.0 ** -12) * mag + (2.0 ** -8 if out == "bf16" else 2.0 ** -24) * np.abs(want)
    assert (np.abs(f64(y) - want) <= bound).all()


# Exact results (float32 queries and results). Units of the last place are 2^-24 of a value.
#   Operands: three bfloat16 terms hold 24 bits, two binary16 terms 22, a weight's exponential 22.
#   A tensor-core sum is cut off at each of its steps of 16 elements; a score of d elements adds up to d / 64
#   sums of 4 steps, and a result's steps are added in fp32, rounded.
@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("heads,dim", [(1, 64), (8, 128), (16, 128), (8, 256), (16, 64), (4, 192)])
@pytest.mark.parametrize("width", [1, 400])
def test_attention_scores_hold_every_term_of_a_query(cache, heads, dim, width):
    """One key: the log-sum-exp is its score, the result its value.

    Query elements are 1 + 2^-9 + 0.9 * 2^-17, so that what a missing term would hold adds up over the elements:
    0.9 * 2^-17 of the score without a third bfloat16 term, 2^-9 without a second binary16 one. Bound, of sum |q k| scale:
    operands 2^-22, the steps of a score 2^-24 each and at most 16 of them (2^-20, all cut the same way), the scale's and
    the logarithm's roundings 4 * 2^-24, and 2^-20 for the shift by the binary16 weights' factor 2^14."""
    g = torch.Generator(DEV).manual_seed(dim + heads)
    k, v = (torch.randn(1, 16, 1, dim, generator=g, device=DEV).abs().to(TORCH[cache]) for _ in range(2))
    q = torch.full((1, heads, dim), 1 + 2.0 ** -9 + 0.9 * 2.0 ** -17, device=DEV)
    q *= 2.0 ** torch.arange(heads, device=DEV)[None, :, None].clamp(max=3)
    out, lse, divided = attend(q, k, v, [[0]], [1], width, out_dtype=torch.float32)
    assert divided == (width > 100 or dim > 128 and width > 1)
    score = (f64(q) * f64(k)[0, 0]).sum(-1) * dim ** -0.5           # all products are positive
    assert (np.abs(f64(lse) - score) <= score * (2.0 ** -20 + 2.0 ** -22 + 2.0 ** -22) + 2.0 ** -20).all()
    assert torch.equal(out[0], v[0, 0].float().expand(heads, dim))


@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("heads,dim", [(1, 64), (8, 128), (16, 128), (8, 256), (16, 64), (4, 192)])
@pytest.mark.parametrize("width", [13, 60, 400])
def test_attention_results_hold_every_term_of_a_weight(cache, heads, dim, width):
    """Equal values are their own average, whatever the weights; weights are 1 and 1/2 + 2^-10 + 0.45 * 2^-17 of it, so that
    what a missing term would hold adds up over the keys.

    Bound: the weights' terms 2^-22, the sums of 16 keys 3 * 2^-24, cut (one for each term), their additions and the sum
    of the weights 2^-24 each, rounded, for at most 13 of a row of 200 keys: 2^-19.2, 2^-19 allowed (a missing third bfloat16
    term is 0.9 * 2^-17, a second binary16 one 2^-12)."""
    k = torch.zeros(13, 16, 1, dim, device=DEV)
    q = torch.zeros(1, heads, dim, device=DEV)
    k[..., 0] = 1.0
    k[0, 0, 0, 0] = 0.0
    q[..., 0] = float(np.log(0.5 + 2.0 ** -10 + 0.45 * 2.0 ** -17) * dim ** 0.5)
    v = torch.full((13, 16, 1, dim), 1.5, device=DEV)
    out, lse, _ = attend(q, k.to(TORCH[cache]), v.to(TORCH[cache]), [list(range(13))], [200], width, out_dtype=torch.float32)
    assert (np.abs(f64(out) - 1.5) <= 1.5 * 2.0 ** -19).all()
    assert np.abs(f64(lse) - np.log(1 + 199 * (0.5 + 2.0 ** -10 + 0.45 * 2.0 ** -17))).max() < 2.0 ** -18


@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
@pytest.mark.parametrize("heads,kvh,dim", [(2, 1, 64), (8, 1, 128), (16, 1, 128), (12, 1, 64), (8, 1, 256), (20, 2, 256), (6, 2, 192)])
@pytest.mark.parametrize("lengths,width", [([190], 13), ([200, 130], 60), ([900], 60), ([2000, 77], 130), ([3000, 1, 20001], 1251)])
def test_attention_exact_results_on_every_path(cache, heads, kvh, dim, lengths, width):
    """float32 results against 64 bits, 2-norm of the whole result, keys, values and queries of unit variance.

    Relative error: weights 2^-22 from the operands' terms and 2^-22 from the exponential, scores 2^-21 (the cut sums of
    scores of about one), each 16 keys' sum 2^-22, and the additions 2^-22: 8e-7 in quadrature, 2^-19 allowed."""
    rng = np.random.default_rng(heads * dim)
    pages = sum(-(-n // 16) for n in lengths)
    k, v = (torch.from_numpy(rng.standard_normal((pages, 16, kvh, dim)).astype(np.float32)).to(DEV).to(TORCH[cache]) for _ in range(2))
    q = torch.from_numpy(rng.standard_normal((len(lengths), heads, dim)).astype(np.float32)).to(DEV)
    table, at = np.full((len(lengths), max(-(-n // 16) for n in lengths)), -1), 0
    for r, n in enumerate(lengths):
        table[r, :-(-n // 16)] = at + np.arange(-(-n // 16))
        at += -(-n // 16)
    out, lse, _ = attend(q, k, v, table, lengths, width, out_dtype=torch.float32)
    for r, n in enumerate(lengths):
        used = torch.from_numpy(table[r, :-(-n // 16)]).to(DEV)
        for h in range(heads):
            keys, values = ((x.float() if cache == "e4m3" else x)[used][:, :, h // (heads // kvh)].reshape(-1, dim)[:n].double() for x in (k, v))
            s = keys @ q[r, h].double() * dim ** -0.5
            want = torch.softmax(s, 0) @ values
            assert (out[r, h].double() - want).norm() <= 2.0 ** -19 * want.norm(), (r, h)
            assert (lse[r, h].double() - torch.logsumexp(s, 0)).abs() <= 2.0 ** -18, (r, h)


# ----------------------------------------------------------------- tables ---
@pytest.mark.parametrize("lengths,new,page,table,status", [
    ([40], None, 16, [[1, 2]], nt.KV_ROW_TOO_SHORT),                       # in a page that the row has no entry for, taking none
    ([16, 33], [0, 15], 16, [[3], [4]], nt.KV_ROW_TOO_SHORT),              # 48 tokens: the row's third page is full, none taken
    ([40], [0], 16, [[1, 2]], 0),                                          # no new token, nothing lost
    ([31], None, 16, [[1, 2]], 0), ([32], None, 16, [[1, 2]], nt.KV_ROW_TOO_SHORT), ([32], [0], 16, [[1, 2]], 0)])
def test_tables_rows_too_short(lengths, new, page, table, status):
    word = torch.zeros(1, dtype=torch.int32, device=DEV)
    t = nt.ninfer_kv_tables(i32(lengths), None if new is None else i32(new), page, i32([9, 8, 7]), i32(table), 20, status=word)
    want = od.kv_tables(lengths, [1] * len(lengths) if new is None else new, page, [9, 8, 7], table, 20)
    for a, b in zip(t, want):
        assert np.array_equal(a.cpu().numpy(), b)
    assert int(word) == want[-1] == status
    assert not status or -1 in t.slots[:int(t.counts[0])].tolist()


def test_tables_of_lengths_that_hold_anything_end_with_their_buffers():
    """The largest new counts for every request (3e11 tokens in all): the work is that of the buffers' sizes."""
    n = 150
    rng = np.random.default_rng(3)
    lengths, new = rng.integers(0, 40, n), np.full(n, 2 ** 31 - 1)
    new[[5, 77]] = 0
    table, free = np.full((n, 6), -1), rng.permutation(800)
    held = -(-lengths // 8)
    table[np.arange(6) < held[:, None]] = 1000 + np.arange(held.sum())
    for capacity in (0, 1, 30, 1000):
        word = torch.zeros(1, dtype=torch.int32, device=DEV)
        t = nt.ninfer_kv_tables(i32(lengths), i32(new), 8, i32(free), i32(table), capacity, status=word)
        torch.cuda.synchronize()
        # page counts run up to 2^28 a request, so that the first request takes the whole list; the others' entries are -1
        want = table.copy()
        for i in range(n):
            if new[i]:
                want[i, held[i]:] = free[:6 - held[i]] if i == 0 else -1
        assert np.array_equal(t.block_table.cpu().numpy(), want), capacity
        assert t.counts.tolist() == [2 ** 31 - 1] * 2
        position = np.arange(lengths[0], lengths[0] + capacity)
        entry = want[0][np.minimum(position // 8, 5)]
        slots = np.where(position // 8 < 6, entry * 8 + position % 8, -1)
        assert np.array_equal(t.slots.cpu().numpy(), slots) and np.array_equal(t.positions.cpu().numpy(), position)
        assert not t.token_rows.any() and t.offsets.tolist()[:2] == [0, 2 ** 31 - 1]
        assert int(word) == nt.KV_OUT_OF_PAGES | nt.KV_ROW_TOO_SHORT | nt.KV_OUT_OF_SLOTS | nt.KV_BAD_LENGTH


@pytest.mark.parametrize("page", [1, 7, 16])
@pytest.mark.parametrize("requests", [3, 1500])
def test_tables_with_fewer_slots_than_tokens(requests, page):
    """Whole tables whatever the slots hold: none of them, the middle of a page or of a request, all but one."""
    rng = np.random.default_rng(requests)
    lengths, new = rng.integers(0, 50, requests), rng.integers(0, 60, requests)
    held, last = -(-lengths // page), -(-(lengths + new) // page)
    pool = rng.permutation(int(last.sum()))
    table = np.full((requests, int(last.max())), -1, np.int64)
    table[np.arange(table.shape[1]) < held[:, None]] = pool[:held.sum()]
    total = int(new.sum())
    for capacity in (0, 1, 5, total // 3, total // 2 + 1, total - 1, total, total + 9):
        for width in (table.shape[1], 3):
            for free in (pool[held.sum():], pool[held.sum():][:20]):
                t = nt.ninfer_kv_tables(i32(lengths), i32(new), page, i32(free), i32(table[:, :width]), capacity)
                for a, b in zip(t, od.kv_tables(lengths, new, page, free, table[:, :width], capacity)):
                    assert np.array_equal(a.cpu().numpy(), b)


def test_tables_outputs_between_a_tables_rows():
    """Lengths in place are refused; what lies between the rows of a wider buffer is no part of the table."""
    wide = torch.full((3, 8), -1, dtype=torch.int32, device=DEV)
    table, lengths, free = wide[:, :5], i32([0, 3, 9]), i32([7, 2, 5])
    out = nt.KvTables.empty(table, 3)
    with pytest.raises(nt.NinferError) as e:
        nt.ninfer_kv_tables(lengths, None, 8, free, table, 3, out=out._replace(lengths=lengths))
    assert e.value.status == 1 and (wide == -1).all()
    t = nt.ninfer_kv_tables(lengths, None, 8, free, table, 3, out=out._replace(counts=wide[1, 5:7]))
    assert wide.tolist() == [[7] + [-1] * 7, [-1] * 5 + [3, 1, -1], [-1] * 8] and t.lengths.tolist() == [1, 4, 10]


def test_tables_and_cache_follow_memory_that_is_replaced():
    """A batch whose rows get more pages, and a cache that gets more of them, in place."""
    table, free = torch.full((2, 2), -1, dtype=torch.int32, device=DEV), i32([3, 1, 0, 2, 7, 6, 5, 4])
    out = nt.KvTables.empty(table, 2)
    nt.ninfer_kv_tables(i32([0, 7]), None, 8, free, table, 2, out=out)
    old = table.detach().clone()
    twin = copy.deepcopy(out)
    nt.ninfer_kv_tables(i32([16, 40]), None, 8, free, twin.block_table, 2, out=twin)
    assert torch.equal(out.block_table, old) and out.lengths.tolist() == [1, 8] and twin.lengths.tolist() == [17, 41]
    table.resize_(2, 6).fill_(-1)
    t = nt.ninfer_kv_tables(i32([16, 40]), None, 8, free, table, 2, out=out)
    assert table.tolist() == [[-1, -1, 3, -1, -1, -1], [-1] * 5 + [1]] and t.slots.tolist() == [24, 8]
    table.data = table.clone().fill_(-1)
    out.slots.data = torch.zeros(2, dtype=torch.int64, device=DEV)
    t = nt.ninfer_kv_tables(i32([16, 40]), None, 8, free, table, 2, out=out)
    assert table.tolist() == [[-1, -1, 3, -1, -1, -1], [-1] * 5 + [1]] and out.slots.tolist() == [24, 8]

    k, v = torch.zeros(2, 8, 1, 16, dtype=torch.bfloat16, device=DEV), torch.zeros(2, 8, 1, 16, dtype=torch.bfloat16, device=DEV)
    cache = nt.KvCache(k, v)
    x = torch.ones(2, 1, 16, dtype=torch.bfloat16, device=DEV)
    nt.ninfer_kv_append(cache, x, x, torch.tensor([3, 15], device=DEV))
    for p in (k, v):
        p.resize_(4, 8, 1, 16)
        p[2:] = 0
    nt.ninfer_kv_append(cache, x * 2, x * 3, t.slots)
    assert (k[3, 0] == 2).all() and (v[1, 0] == 3).all() and (k[0, 3] == 1).all() and (k[1, 7] == 1).all()
    y = nt.ninfer_kv_attention(x[:, :, :16].contiguous(), cache, i32([[3], [1]]), i32([1, 1]))
    assert torch.equal(y[0], v[3, 0]) and (y[1] == 3).all()


# ----------------------------------------------------------------- append ---
@pytest.mark.parametrize("scale", [0.0137, 0.0625, 0.31, 1.7, 3.0, 2.0 ** -130, 1e30])
@pytest.mark.parametrize("src", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("cache", ["bf16", "f16", "e4m3"])
def test_append_rounds_the_quotient_once(cache, src, scale):
    """Sources whose quotients lie at, just below and just above the points halfway between two values of the cache's type.

    The quotient in 64 bits decides: a quotient of two 24-bit numbers that is not halfway between two values
    of at most 8 bits (11 of f16) differs from that point by more than 2^-24 * 2^-12 of itself, which 53 bits show."""
    rng = np.random.default_rng(7)
    scale = float(np.float32(scale))
    bits = {"bf16": 8, "f16": 11, "e4m3": 4}[cache]
    halfway = (2 * rng.integers(2 ** (bits - 1), 2 ** bits, 6000) + 1) * 2.0 ** rng.integers(-24, 4, 6000) * rng.choice([-1, 1], 6000)
    halfway[::7] = rng.standard_normal(halfway[::7].size) * 30
    with np.errstate(over="ignore"):
        x = torch.from_numpy((halfway * scale).astype(np.float32)).to(TORCH[src])
    x[:16] = torch.tensor([0.0, -0.0, float("inf"), -float("inf"), float("nan"), 3e38, -3e38, 1e-45, -1e-45, 1e-38, 65504.0, 1.0,
                           448.0, 464.0, 1e-4, -6e-8]).to(TORCH[src])
    x = x.view(375, 1, 16)
    k, v = (torch.zeros(24, 16, 1, 16, device=DEV).to(TORCH[cache]) for _ in range(2))
    nt.ninfer_kv_append(nt.KvCache(k, v, scale, 1.0), x.to(DEV), x.to(DEV), torch.arange(375, device=DEV))
    for pool, by in ((k, scale), (v, 1.0)):
        want = od.round_to(f64(x) / by, cache, cache == "e4m3").reshape(-1)
        if cache == "e4m3":
            want = np.where(np.isinf(f64(x).reshape(-1)), np.sign(f64(x).reshape(-1)) * 448.0, want)
        got = f64(pool).reshape(-1)[:want.size]
        assert np.array_equal(got, want, equal_nan=True), np.argwhere(got != want)[:5]
        assert np.array_equal(np.signbit(got[got == 0]), np.signbit(want[got == 0]))


# ----------------------------------------------------------------- logits ---
def test_logits_bias_offsets_are_cut_at_both_ends():
    """Offsets past bias_count, up to the largest int32, and negative ones: nothing is read there."""
    x = torch.randn(6, 700, device=DEV)
    offsets = i32([2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 200, -2 ** 31, 2, 2 ** 31 - 1, 1])
    ids, values = i32([5, 600, 7]), torch.tensor([1.0, 2.0, 4.0], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    y = nt.ninfer_logits_process(x, bias_offsets=offsets, bias_ids=ids, bias_values=values, status=status)
    want = x.clone()
    want[3, 5] += 1.0           # from -2^31 to 2: the first two entries
    want[3, 600] += 2.0
    want[4, 7] += 4.0           # from 2 to past the end: the last one
    assert torch.equal(y, want) and int(status) == 0


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("vocab", [4096, 4099])
def test_logits_repetitions_without_a_reciprocal(dtype, vocab):
    """Repetitions whose reciprocal is no normal fp32 number: one rounding of the quotient, then of the type."""
    rng = np.random.default_rng(vocab)
    rep = np.array([1e-39, 3e38, 0.0, float("inf"), 1e-45, 2.0 ** 127], np.float32)
    x = torch.from_numpy(rng.standard_normal((6, vocab)).astype(np.float32)).to(DEV)
    x[0] *= 1e-38
    x[4] *= 1e-44
    x[5] *= 2.0 ** 100
    x = x.to(TORCH[dtype])
    h = torch.arange(vocab, dtype=torch.int32, device=DEV).expand(6, vocab).contiguous()
    y = nt.ninfer_logits_process(x, history=h, history_lengths=i32([vocab] * 6), repetition=torch.from_numpy(rep).to(DEV))
    x64, r64 = f64(x), rep.astype(np.float64)[:, None]
    with np.errstate(all="ignore"):
        want = od.round_to(np.where(x64 > 0, x64 / r64, x64 * r64), "f32")
        want = want if dtype == "f32" else od.round_to(want, dtype)
    assert np.array_equal(f64(y), want, equal_nan=True)
