"""Decode-step operators on the GPU against their fp64 definitions.

Bounds, fixed from the number formats:
- tables: whole numbers, equal; append: the stored value is the fp64 quotient
  rounded once, equal (for scale 1 and powers of two; an fp32 quotient that is
  not exact may round a tie the other way: one step there).
- attention: fp32 queries, and the weights of fp32 results, hold 22 bits or more
  in the tensor cores, other weights 16 (bfloat16 caches), and 11 where a
  bfloat16 result comes of a binary16 or 8-bit cache; everything else is fp32. A
  score is then off by at most S 2^-15 with S = scale * sum |q_d k_d| of the row,
  a weight by twice that and its own rounding, W = 2^-15 or 2^-12, and the result by
  (2 S 2^-15 + W) sum_j p_j |v_j|, plus half a step of the output's format.
  lse: (S + |lse| + 1) 2^-15.
- logits: three fp32 roundings of values up to the largest one that a token's
  chain holds, then one of the output's format.
"""
import ctypes as C

import numpy as np
import pytest
import torch

import bit_gemv_gb300 as nt
from oracle import decode as od

pytestmark = pytest.mark.gpu
DEV = torch.device("cuda:0")
TORCH = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
STEP = {"f32": 2.0 ** -24, "bf16": 2.0 ** -8, "f16": 2.0 ** -11}


def f64(t):
    return t.float().cpu().numpy().astype(np.float64)


def i32(a):
    return torch.from_numpy(np.ascontiguousarray(a, np.int32)).to(DEV)


# ----------------------------------------------------------------- tables ---
def run_tables(lengths, new, page, free, table, capacity, pad=0):
    wide = np.full((len(lengths), np.shape(table)[1] + pad), -7, np.int32)
    wide[:, :np.shape(table)[1]] = table
    td = i32(wide)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    view = td[:, :np.shape(table)[1]]
    got = nt.ninfer_kv_tables(i32(lengths), None if new is None else i32(new), page, i32(free) if len(free) else None, view,
                              capacity, status=status)
    first = [t.cpu().numpy().copy() for t in got]
    again = nt.ninfer_kv_tables(i32(lengths), None if new is None else i32(new), page, i32(free) if len(free) else None, view,
                                capacity, out=got)
    for a, b in zip(first, again):
        assert np.array_equal(a, b.cpu().numpy()), "a second call changed something"
    assert (td[:, np.shape(table)[1]:] == -7).all(), "wrote past the row"
    return first, int(status)


def check_tables(lengths, new, page, free, table, capacity, pad=0):
    got, status = run_tables(lengths, new, page, free, table, capacity, pad)
    want = od.kv_tables(lengths, [1] * len(lengths) if new is None else new, page, free, table, capacity)
    for name, a, b in zip(nt.KvTables._fields, got, want):
        assert np.array_equal(a, b), name
    assert status == want[-1]


def random_tables(rng, requests, page, longest, most_new, width_extra=2):
    lengths = rng.integers(0, longest + 1, requests)
    new = rng.integers(0, most_new + 1, requests)
    held, last = -(-lengths // page), -(-(lengths + new) // page)
    pool = rng.permutation(int(last.sum()) + 5)
    table = np.full((requests, int(last.max(initial=0)) + width_extra), -1, np.int64)
    table[np.arange(table.shape[1]) < held[:, None]] = pool[:held.sum()]
    return lengths, new, pool[held.sum():], table


@pytest.mark.parametrize("requests,page,longest,most_new,slack", [
    (1, 16, 0, 1, 0), (1, 16, 40, 1, 3), (3, 1, 9, 5, 0), (64, 16, 900, 1, 0), (64, 16, 0, 300, 17), (33, 24, 500, 100, 1),
    (7, 1000, 5000, 3000, 2), (1023, 8, 60, 3, 0), (1024, 8, 60, 3, 5), (1025, 8, 60, 3, 0), (5000, 16, 40, 2, 100),
    (200, 32, 3, 0, 4)])
def test_tables(requests, page, longest, most_new, slack):
    rng = np.random.default_rng(requests * 31 + page)
    lengths, new, free, table = random_tables(rng, requests, page, longest, most_new)
    check_tables(lengths, new, page, free, table, int(new.sum()) + slack, pad=3)


def test_tables_one_token_each_without_a_list():
    rng = np.random.default_rng(5)
    lengths, _, free, table = random_tables(rng, 40, 16, 300, 1)
    check_tables(lengths, None, 16, free, table, 40)


def test_tables_that_run_out():
    rng = np.random.default_rng(6)
    lengths, new, free, table = random_tables(rng, 20, 8, 100, 60)
    check_tables(lengths, new, 8, free[:len(free) // 3], table, int(new.sum()))             # out of pages
    check_tables(lengths, new, 8, [], table, int(new.sum()))                                 # no page at all
    check_tables(lengths, new, 8, free, table[:, :9], int(new.sum()))                        # rows too short
    check_tables(lengths, new, 8, free, table, int(new.sum()) // 2)                          # too few slots
    check_tables(lengths, new, 8, free, table, 0)
    check_tables([-3, 5, 2], [2, -1, 3], 4, [9, 8, 7, 6], [[-1, -1], [0, 1], [2, -1]], 8)   # negative lengths


def test_tables_outputs_are_optional():
    t = i32(np.full((2, 3), -1))
    assert nt._lib.ninfer_kv_tables(i32([0, 0]).data_ptr(), i32([5, 6]).data_ptr(), 2, 4, i32([4, 3, 2, 1]).data_ptr(), 4,
                                    t.data_ptr(), 3, 3, None, None, None, 0, None, None, None, None, None) == 0
    torch.cuda.synchronize()
    assert t.tolist() == [[4, 3, -1], [2, 1, -1]]


# ----------------------------------------------------------------- append ---
def make_pool(pages, page, heads, dim, dtype, layout, fill=0.0):
    shape = {"tokens": (pages, page, heads, dim), "heads": (pages, heads, page, dim), "inside": (pages, page, 2, heads, dim)}[layout]
    t = torch.full(shape, fill, device=DEV).to(TORCH[dtype])
    return t if layout == "tokens" else t.permute(0, 2, 1, 3) if layout == "heads" else t[:, :, 1]


@pytest.mark.parametrize("layout", ["tokens", "heads", "inside"])
@pytest.mark.parametrize("src", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("dtype,heads,dim,page,tokens,scale", [
    ("bf16", 1, 8, 1, 1, 1.0), ("bf16", 4, 128, 16, 70, 1.0), ("f16", 3, 80, 24, 33, 0.5), ("f16", 16, 256, 64, 129, 1.0),
    ("e4m3", 2, 16, 16, 5, 1.0), ("e4m3", 5, 240, 7, 61, 0.25)])
def test_append(layout, src, dtype, heads, dim, page, tokens, scale):
    rng = np.random.default_rng(tokens + dim)
    pages = -(-tokens // page) + 3
    k, v = (make_pool(pages, page, heads, dim, dtype, layout, 3.0) for _ in range(2))
    rows = torch.from_numpy(rng.standard_normal((tokens, 3, heads, dim)).astype(np.float32) * 60).to(DEV).to(TORCH[src])
    rows.view(-1)[::97] *= 1e4                      # some past the 8-bit range and float16's
    slots = rng.permutation(pages * page)[:tokens]
    skipped = rng.random(tokens) < 0.1
    given = np.where(skipped, -1 - rng.integers(0, 5, tokens), slots)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    cache = nt.KvCache(k, v, scale, scale * 2)
    nt.ninfer_kv_append(cache, rows[:, 1], rows[:, 2], torch.from_numpy(given).to(DEV), status=status)
    assert int(status) == 0
    for pool, j, s in ((k, 1, scale), (v, 2, scale * 2)):
        want = np.full((pages, page, heads, dim), od.round_to(3.0, dtype))
        x = od.round_to(f64(rows[:, j]) / s, "f32")
        want[slots[~skipped] // page, slots[~skipped] % page] = od.round_to(x, dtype, dtype == "e4m3")[~skipped]
        assert np.array_equal(f64(pool), want)


def test_append_bad_slots_and_nan():
    k = torch.zeros(2, 4, 1, 16, dtype=TORCH["e4m3"], device=DEV)
    v = torch.zeros_like(k)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x = torch.full((3, 1, 16), float("nan"), device=DEV)
    x[1] = float("inf")
    nt.ninfer_kv_append(nt.KvCache(k, v), x, x, torch.tensor([7, 2, 8], device=DEV), status=status)
    assert int(status) == nt.KV_BAD_SLOT
    assert torch.isnan(k.float()[1, 3]).all() and (k.float()[0, 2] == 448).all() and int((k.float() != 0).sum()) == 32
    nt.ninfer_kv_append(nt.KvCache(k, v), x, x, torch.tensor([2 ** 40, -2 ** 62, -1], device=DEV))   # no status word, nothing written
    assert int((v.float() != 0).sum()) == 32


# -------------------------------------------------------------- attention ---
def attention_case(rng, lengths, heads, kvh, dim, page, cache="bf16", q="bf16", layout="tokens", spread=1.0, stale=float("nan"),
                   scales=(1.0, 1.0), extra=2):
    """Pools whose every entry outside the requests' tokens is `stale`."""
    lengths = np.asarray(lengths, np.int64)
    used = -(-np.maximum(lengths, 0) // page)
    pages = int(used.sum()) + extra
    pool = rng.permutation(pages)
    table = np.full((len(lengths), max(1, int(used.max(initial=0))) + 1), -1, np.int64)
    table[np.arange(table.shape[1]) < used[:, None]] = pool[:used.sum()]
    kv = []
    for i in range(2):
        t = make_pool(pages, page, kvh, dim, cache, layout, stale)
        x = torch.from_numpy(rng.standard_normal((int(lengths.clip(0).sum()), kvh, dim)).astype(np.float32)).to(DEV)
        x = (x / scales[i]).to(t.dtype)
        pos = np.concatenate([np.arange(max(0, n)) for n in lengths]) if lengths.clip(0).sum() else np.zeros(0, np.int64)
        row = np.repeat(np.arange(len(lengths)), lengths.clip(0))
        at = torch.from_numpy(table[row, pos // page]).to(DEV), torch.from_numpy(pos % page).to(DEV)
        if cache == "e4m3":
            t.view(torch.uint8)[at] = x.view(torch.uint8)
        else:
            t[at] = x
        kv.append(t)
    qq = torch.from_numpy(rng.standard_normal((len(lengths), heads, dim)).astype(np.float32) * spread).to(DEV).to(TORCH[q])
    return qq, kv[0], kv[1], table, lengths


def check_attention(q, k, v, table, lengths, scale=None, window=0, out="bf16", scales=(1.0, 1.0), workspace=None):
    scale = q.shape[2] ** -0.5 if scale is None else scale
    cache = nt.KvCache(k, v, *scales)
    lse = torch.full(q.shape[:2], 7.0, device=DEV)
    y = torch.full(q.shape, float("nan"), device=DEV).to(TORCH[out])
    nt.ninfer_kv_attention(q, cache, i32(table), i32(lengths), scale=scale, window=window, out=y, lse=lse, workspace=workspace)
    torch.cuda.synchronize()
    assert nt.ninfer_device_errors() == 0
    want, wlse, mag, big = od.kv_attention(f64(q), f64(k), f64(v), table, lengths, scale, window, *scales)
    got, glse = f64(y), f64(lse)
    weight = 2.0 ** -12 if out == "bf16" and k.dtype != torch.bfloat16 else 2.0 ** -15
    bound = (2 * big[..., None] * 2.0 ** -15 + weight) * mag + STEP[out] * np.abs(want) + (2.0 ** -25 if out == "f16" else 0)
    bad = ~(np.abs(got - want) <= bound)
    assert not bad.any(), (np.argwhere(bad)[:5], got[bad][:5], want[bad][:5])
    empty = wlse == -np.inf
    assert (glse[empty] == -np.inf).all()
    glse, wlse = np.where(empty, 0, glse), np.where(empty, 0, wlse)
    assert (np.abs(glse - wlse)[~empty] <= ((big + np.abs(wlse) + 1) * 2.0 ** -15)[~empty]).all()
    return y


@pytest.mark.parametrize("cache,q,out", [("bf16", "bf16", "bf16"), ("f16", "f16", "f16"), ("e4m3", "bf16", "bf16"),
                                         ("bf16", "f32", "f32"), ("f16", "f32", "f32"), ("e4m3", "f32", "f32"),
                                         ("f16", "bf16", "f32"), ("bf16", "f16", "bf16")])
@pytest.mark.parametrize("heads,kvh,dim,page,layout", [
    (8, 1, 128, 16, "tokens"), (6, 1, 256, 64, "heads"), (24, 4, 256, 16, "tokens"), (4, 4, 64, 24, "heads"),
    (5, 5, 16, 1, "tokens"), (9, 1, 80, 3, "inside"), (32, 2, 112, 7, "heads"), (20, 1, 192, 100, "tokens"),
    (14, 2, 48, 2, "inside"), (2, 1, 240, 512, "heads")])
def test_attention_heads_pages_and_types(cache, q, out, heads, kvh, dim, page, layout):
    rng = np.random.default_rng(heads * 1000 + dim)
    lengths = [0, 1, 2, 15, 16, 17, 33, 64, 65, 131, 300]
    scales = (0.125, 0.0625) if cache == "e4m3" else (1.0, 1.0)
    case = attention_case(rng, lengths, heads, kvh, dim, page, cache, q, layout, 1.5, scales=scales)
    check_attention(*case, out=out, scales=scales)


@pytest.mark.parametrize("window", [1, 2, 31, 32, 33, 64, 100, 299, 300, 5000])
@pytest.mark.parametrize("cache,dim,page", [("bf16", 128, 16), ("e4m3", 64, 24), ("f16", 256, 1)])
def test_attention_window(window, cache, dim, page):
    rng = np.random.default_rng(window)
    check_attention(*attention_case(rng, [0, 1, 31, 32, 33, 64, 65, 300, 301], 6, 2, dim, page, cache, "bf16"), window=window)


@pytest.mark.parametrize("dim", [8, 24, 40, 56, 72, 88, 136, 200, 248])
def test_attention_head_dims(dim):
    rng = np.random.default_rng(dim)
    check_attention(*attention_case(rng, [1, 40, 77], 6, 2, dim, 16, "bf16", "f32"), out="f32")
    check_attention(*attention_case(rng, [1, 40, 77], 3, 3, dim, 16, "f16", "f16", "heads"), out="f16")


@pytest.mark.parametrize("heads,kvh", [(1, 1), (7, 7), (8, 8), (16, 1), (17, 1), (64, 1), (40, 8)])
def test_attention_groups(heads, kvh):
    rng = np.random.default_rng(heads)
    check_attention(*attention_case(rng, [5, 90, 257], heads, kvh, 64, 16, "bf16", "bf16"))


@pytest.mark.parametrize("heads,kvh,dim", [(9, 1, 128), (24, 2, 64), (16, 1, 104), (33, 1, 128), (16, 1, 136), (44, 2, 256)])
@pytest.mark.parametrize("cache,q,out", [("bf16", "bf16", "bf16"), ("bf16", "f32", "f32"), ("f16", "f16", "bf16"),
                                         ("e4m3", "bf16", "bf16"), ("e4m3", "f32", "f32")])
def test_attention_wide_groups_split_and_joined(heads, kvh, dim, cache, q, out):
    """Sixteen heads to a row, a last row of fewer, in rows that are cut between warps and CTAs."""
    rng = np.random.default_rng(heads + dim)
    dim = dim // 16 * 16 if cache == "e4m3" else dim
    check_attention(*attention_case(rng, [6001, 3, 0, 777], heads, kvh, dim, 16, cache, q, "heads"), out=out)


@pytest.mark.parametrize("lengths,heads,kvh,dim,page,cache", [
    ([70001], 8, 1, 128, 16, "bf16"), ([9001], 4, 2, 64, 64, "f16"), ([20011, 3, 0, 5000], 6, 1, 256, 32, "bf16"),
    ([30011], 2, 1, 128, 1, "e4m3"), ([1] * 500, 4, 2, 128, 16, "bf16"), (list(range(300)), 2, 2, 64, 8, "f16"),
    ([0] * 2000 + [50], 4, 1, 64, 16, "bf16"), ([0, 0], 4, 1, 64, 16, "bf16"), ([1500] * 12, 8, 4, 128, 16, "e4m3"),
    ([7, 0] * 1300, 2, 1, 64, 16, "bf16")])
def test_attention_split_and_joined(lengths, heads, kvh, dim, page, cache):
    rng = np.random.default_rng(len(lengths))
    check_attention(*attention_case(rng, lengths, heads, kvh, dim, page, cache, "bf16", spread=2.0))


@pytest.mark.parametrize("seed", range(24))
def test_attention_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    cache = str(rng.choice(["bf16", "f16", "e4m3"]))
    kvh, group = int(rng.integers(1, 9)), int(rng.integers(1, 13))
    dim = int(rng.integers(1, 17)) * (16 if cache == "e4m3" else 8)
    page = int(rng.choice([1, 3, 8, 16, 20, 32, 48, 64, 128, 129]))
    lengths = np.exp(rng.uniform(0, np.log(4000), int(rng.integers(1, 20)))).astype(int) - 1
    scales = (0.25, 0.125) if cache == "e4m3" else (1.0, 1.0)
    case = attention_case(rng, lengths, kvh * group, kvh, dim, page, cache, str(rng.choice(["f32", "bf16", "f16"])),
                          str(rng.choice(["tokens", "heads", "inside"])), 1.5, scales=scales)
    check_attention(*case, window=int(rng.choice([0, 0, 1, 700])), out=str(rng.choice(["f32", "bf16", "f16"])), scales=scales)


def test_attention_extreme_scores():
    rng = np.random.default_rng(3)
    for cache, top in (("bf16", 3e38), ("f16", 65504.0), ("e4m3", 448.0)):
        q, k, v, table, lengths = attention_case(rng, [200, 200, 200, 200], 4, 1, 64, 16, cache, "f32", stale=0.0)
        flat = torch.arange(200, device=DEV)
        for r in range(4):
            page = torch.from_numpy(table[r]).to(DEV)[flat // 16]
            # rising and falling scores (a new maximum at every key, or none after the first), up to +-400; then the type's largest
            x = {0: flat * 2.0, 1: -flat * 2.0, 2: torch.where(flat % 7 == 0, 50.0, -50.0), 3: flat * 0 + 400.0}[r]
            kk = torch.zeros(200, 1, 64, device=DEV)
            kk[:, 0, 0] = x
            (k.view(torch.uint8) if cache == "e4m3" else k)[page, flat % 16] = \
                kk.to(k.dtype).view(torch.uint8) if cache == "e4m3" else kk.to(k.dtype)
        q.zero_()
        q[:, :, 0] = 1.0
        check_attention(q, k, v, table, lengths, scale=1.0, out="f32")
        # queries and keys at the type's lowest value: one key far below, or far above, all others
        q[:, :, 0] = 1e-3
        kk = k.float()
        kk[table[0][0], 3, 0, 0] = -top
        kk[table[1][0], 3, 0, 0] = top
        check_attention(q, kk.clamp(-top, top).to(k.dtype), v, table, lengths, scale=1.0, out="f32")


def test_attention_large_and_small_queries():
    """Queries far outside float16's range against float16 and 8-bit keys."""
    rng = np.random.default_rng(4)
    for cache in ("f16", "e4m3", "bf16"):
        q, k, v, table, lengths = attention_case(rng, [100, 37], 4, 2, 64, 16, cache, "f32")
        for factor in (1e7, 1e-7, 1e20):
            check_attention(q * factor, k, v, table, lengths, scale=0.125 / factor, out="f32")
    q.zero_()
    check_attention(q, k, v, table, lengths, out="f32")


def test_attention_scores_of_minus_infinity():
    """Keys that score -infinity have no weight; a row of nothing else is empty."""
    rng = np.random.default_rng(5)
    q, k, v, table, lengths = attention_case(rng, [50, 50], 2, 1, 64, 16, "f16", "f16", stale=0.0)
    q.zero_()
    q[:, :, 0] = 1.0
    k.zero_()
    k[table[0][0], 0:5, 0, 0] = -float("inf")
    for p in table[1][:4]:
        k[p, :, 0, 0] = -float("inf")
    cache, lse = nt.KvCache(k, v), torch.zeros(2, 2, device=DEV)
    y = nt.ninfer_kv_attention(q, cache, i32(table), i32(lengths), scale=1.0, lse=lse, out_dtype=torch.float32)
    rows = np.concatenate([f64(v)[table[0][j // 16], j % 16, 0][None] for j in range(5, 50)])
    assert np.allclose(f64(y)[0], rows.mean(0), atol=2e-5) and np.allclose(f64(lse)[0], np.log(45), atol=1e-5)
    assert (y[1] == 0).all() and (lse[1] == -float("inf")).all()


def test_attention_weights_far_below_the_largest():
    """Many keys whose weights lie far under one key's still count."""
    n = 60000
    k = torch.zeros(n // 16, 16, 1, 64, dtype=torch.float16, device=DEV)
    v = torch.ones_like(k)
    k[0, 0, 0, 0] = 17.0                     # e^17 = 2.4e7 against 60000 weights of 1
    v[0, 0] = -1.0
    q = torch.zeros(1, 1, 64, dtype=torch.float32, device=DEV)
    q[..., 0] = 1.0
    check_attention(q, k, v, np.arange(n // 16)[None], [n], scale=1.0, out="f32")
    check_attention(q, k.to(torch.float8_e4m3fn), v.to(torch.float8_e4m3fn), np.arange(n // 16)[None], [n], scale=1.0, out="f32")


def test_attention_table_entries_outside_the_pool():
    """Bad entries beyond a request's length are never read; within it they stand for zeros; lengths past the table are cut."""
    rng = np.random.default_rng(6)
    q, k, v, table, lengths = attention_case(rng, [40, 90, 16], 4, 2, 64, 16, "bf16", "f32", stale=0.0)
    table[0, 3:], table[2, 1:] = 2 ** 31 - 1, -2 ** 31
    check_attention(q, k, v, table, lengths, out="f32")
    table[1, 2], table[1, 4] = 10 ** 6, -5
    check_attention(q, k, v, table, lengths, out="f32")
    check_attention(q, k, v, table[:, :2].copy(), [2 ** 31 - 1, 90, -7], out="f32")


def test_attention_strided_queries_and_tables():
    rng = np.random.default_rng(7)
    q, k, v, table, lengths = attention_case(rng, [40, 90, 16], 6, 2, 64, 16, "bf16", "bf16")
    fused = torch.randn(3, 10, 128, device=DEV, dtype=torch.bfloat16)        # q with gates between its heads, and more behind
    fused[:, :6, :64] = q
    wide = np.full((3, table.shape[1] + 5), 77, np.int64)
    wide[:, :table.shape[1]] = table
    td, cache = i32(wide), nt.KvCache(k, v)
    a = nt.ninfer_kv_attention(fused[:, :6, :64], cache, td[:, :table.shape[1]], i32(lengths))
    b = nt.ninfer_kv_attention(q, cache, i32(table), i32(lengths))
    assert torch.equal(a, b)


def test_attention_offsets_past_32_bits():
    """Pages whose bytes lie past 4 GiB, and whose elements lie past 2^31."""
    for cache in ("e4m3", "bf16"):
        pages = 40000
        k = torch.empty(pages, 16, 8, 1024 // 8, dtype=torch.uint8 if cache == "e4m3" else torch.bfloat16, device=DEV)
        v = torch.empty_like(k)
        k, v = (t.view(torch.float8_e4m3fn) if cache == "e4m3" else t for t in (k, v))
        table = np.array([[pages - 1, 0, pages - 2, 35001], [7, 38000, 9, 39000]])
        g = torch.Generator(DEV).manual_seed(1)
        for t in (k, v):
            for p in table.reshape(-1):
                t[p] = torch.randn(16, 8, 128, generator=g, device=DEV).to(t.dtype)
        q = torch.randn(2, 16, 128, generator=g, device=DEV)
        small = [torch.stack([t[p] for p in table.reshape(-1)]) if cache != "e4m3" else
                 torch.stack([t.view(torch.uint8)[p] for p in table.reshape(-1)]).view(t.dtype) for t in (k, v)]
        a = nt.ninfer_kv_attention(q, nt.KvCache(k, v), i32(table), i32([64, 55]))
        b = check_attention(q, small[0], small[1], np.arange(8).reshape(2, 4), [64, 55], out="f32")
        assert torch.equal(a, b)
        # and the append reaches them
        x = torch.ones(1, 8, 128, device=DEV)
        nt.ninfer_kv_append(nt.KvCache(k, v), x, x, torch.tensor([(pages - 1) * 16 + 15], device=DEV))
        assert (k[pages - 1, 15].float() == 1).all() and (v[pages - 1, 15].float() == 1).all()
        del k, v


def test_attention_streams_graphs_and_one_workspace():
    """Several shapes through one workspace, on a side stream and replayed in a graph: equal to the plain calls."""
    rng = np.random.default_rng(8)
    cases = [attention_case(rng, ls, 8, 2, 128, 16, "bf16", "bf16") for ls in ([5000, 3], [1] * 40, [700] * 9)]
    caches = [nt.KvCache(c[1], c[2]) for c in cases]
    tables, lengths = [i32(c[3]) for c in cases], [i32(c[4]) for c in cases]
    need = max(nt.ninfer_kv_attention_workspace(h, len(c[4]), 8) for h, c in zip(caches, cases))
    want = [nt.ninfer_kv_attention(c[0], h, t, n) for c, h, t, n in zip(cases, caches, tables, lengths)]
    ws = torch.randint(0, 255, (need + 1,), dtype=torch.uint8, device=DEV)
    out = [torch.empty_like(w) for w in want]

    def all_of_them():
        for c, h, t, n, o in zip(cases, caches, tables, lengths, out):
            nt.ninfer_kv_attention(c[0], h, t, n, out=o, workspace=ws)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        all_of_them()
    stream.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(out, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        all_of_them()
    for _ in range(3):
        for o in out:
            o.fill_(float("nan"))
        ws.random_(0, 255)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_attention_is_deterministic():
    rng = np.random.default_rng(9)
    q, k, v, table, lengths = attention_case(rng, [20000, 17, 900], 8, 1, 128, 16, "bf16", "f32")
    cache = nt.KvCache(k, v)
    a = [nt.ninfer_kv_attention(q, cache, i32(table), i32(lengths), out_dtype=torch.float32) for _ in range(4)]
    assert all(torch.equal(a[0], x) for x in a)


# ----------------------------------------------------------------- logits ---
def check_logits(rng, rows, vocab, dtype="f32", longest=0, prompts=True, penalties="rpf", biases=0, masks=0, mask_rows=True,
                 in_place=False, pad=0, offset=0):
    kw, ok = {}, {}
    x = torch.from_numpy(rng.standard_normal((rows, vocab + pad)).astype(np.float32) * 5).to(DEV).to(TORCH[dtype])[:, :vocab]
    if longest:
        h = (vocab * rng.random((rows, longest)) ** 4).astype(np.int64)
        n = rng.integers(0, longest + 1, rows)
        n[0] = longest
        ok.update(history=h, history_lengths=n)
        kw.update(history=i32(h), history_lengths=i32(n))
        if prompts:
            ok["prompt_lengths"] = rng.integers(0, longest + 1, rows)
            kw["prompt_lengths"] = i32(ok["prompt_lengths"])
    for c, name, low, high in (("r", "repetition", 0.8, 1.5), ("p", "presence", -1, 1), ("f", "frequency", -0.2, 0.4)):
        if c in penalties:
            a = rng.uniform(low, high, rows).astype(np.float32)
            ok[name], kw[name] = a, torch.from_numpy(a).to(DEV)
    if biases:
        each = rng.integers(0, min(biases, vocab) + 1, rows)
        ids = [rng.choice(vocab, e, replace=False) for e in each]
        vals = rng.normal(0, 3, each.sum()).astype(np.float32)
        at = np.concatenate([[0], np.cumsum(each)])
        ok["bias"] = [dict(zip(ids[b].tolist(), vals[at[b]:at[b + 1]].tolist())) for b in range(rows)]
        kw.update(bias_offsets=i32(at), bias_ids=i32(np.concatenate(ids)), bias_values=torch.from_numpy(vals).to(DEV))
    if masks:
        words = -(-vocab // 32) + 1
        m = rng.integers(0, 2 ** 32, (masks, words), dtype=np.uint64).astype(np.uint32)
        ok["mask"] = np.unpackbits(m.view(np.uint8).reshape(masks, -1), axis=1, bitorder="little")[:, :vocab].astype(bool)
        kw["mask"] = torch.from_numpy(m.view(np.int32)).to(DEV)
        if mask_rows:
            ok["mask_rows"] = rng.integers(-1, masks, rows)
            kw["mask_rows"] = i32(ok["mask_rows"])
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    x64 = f64(x)
    got = f64(nt.ninfer_logits_process(x, out=x if in_place else None, status=status, **kw))
    want = od.logits_process(x64, **ok)
    assert int(status) == 0
    assert np.array_equal(got == -np.inf, want == -np.inf)
    f = np.isfinite(want)
    got, want = np.where(f, got, 0), np.where(f, want, 0)
    chain = 100.0 + np.abs(want)            # values on the way: logits to 30, penalties to 0.4 * count, biases to 15
    if longest:
        chain = chain + longest
    assert (np.abs(got - want)[f] <= (chain * 2.0 ** -22 + STEP[dtype] * np.abs(want))[f]).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("rows,vocab,pad", [(1, 1, 0), (2, 31, 1), (3, 33, 0), (1, 8192, 0), (5, 8193, 8), (2, 50257, 3),
                                            (1, 248320, 0), (3, 70001, 0), (9, 1000, 24)])
def test_logits(dtype, rows, vocab, pad):
    rng = np.random.default_rng(vocab)
    check_logits(rng, rows, vocab, dtype, longest=200, biases=20, masks=2, pad=pad)
    check_logits(rng, rows, vocab, dtype, longest=50, biases=5, masks=3, in_place=True, pad=pad)


@pytest.mark.parametrize("kw", [dict(), dict(longest=9), dict(longest=9, penalties=""), dict(longest=30, penalties="r", prompts=False),
                                dict(longest=30, penalties="p"), dict(longest=30, penalties="f"), dict(biases=40), dict(masks=4),
                                dict(masks=6, mask_rows=False), dict(longest=5000, penalties="rpf"), dict(longest=1, biases=1)])
def test_logits_parts(kw):
    check_logits(np.random.default_rng(2), 4, 4099, **kw)


def test_logits_one_token_many_times():
    n, vocab = 200000, 300
    x = torch.ones(1, vocab, device=DEV)
    h = torch.full((1, n), 7, dtype=torch.int32, device=DEV)
    y = nt.ninfer_logits_process(x, history=h, history_lengths=i32([n]), prompt_lengths=i32([5]),
                                 frequency=torch.tensor([0.5], device=DEV))
    assert y[0, 7] == 1 - 0.5 * (n - 5) and int((y != 1).sum()) == 1


def test_logits_bad_tokens_and_special_values():
    x = torch.tensor([[float("nan"), float("inf"), -float("inf"), -2.0, 3.0, 3.4e38, -3.4e38, 0.0]], device=DEV)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    h = i32([[-1, 8, 2 ** 31 - 1, 0, 1, 2, 5, 6]])
    y = nt.ninfer_logits_process(x, history=h, history_lengths=i32([8]), repetition=torch.tensor([2.0], device=DEV),
                                 bias_offsets=i32([0, 3]), bias_ids=i32([9, -1, 4]),
                                 bias_values=torch.tensor([1.0, 1.0, 4.0], device=DEV), status=status)
    assert int(status) == nt.LOGITS_BAD_TOKEN
    got = y[0].tolist()
    assert got[0] != got[0] and got[1:3] == [float("inf"), -float("inf")] and got[3:5] == [-2.0, 7.0] and got[7] == 0.0
    assert got[5] == float(torch.tensor(3.4e38) / 2) and got[6] == -float("inf")       # -3.4e38 * 2 is past fp32
    status.zero_()
    nt.ninfer_logits_process(x, mask=i32([[0]]), mask_rows=i32([1]), status=status)     # a mask row past the last: no mask
    assert int(status) == nt.LOGITS_BAD_TOKEN
    y = nt.ninfer_logits_process(x, mask=i32([[0]]), mask_rows=i32([0]))                # everything forbidden, NaN too
    assert (y == -float("inf")).all()
    lengths = nt.ninfer_logits_process(x, history=h, history_lengths=i32([99]), repetition=torch.tensor([2.0], device=DEV))
    assert torch.equal(torch.nan_to_num(lengths[0, 5:]), torch.nan_to_num(y.new_tensor([1.7e38, -float("inf"), 0.0])))


# ---------------------------------------------------------------- refusals ---
def test_device_refusals():
    k = torch.zeros(3, 4, 2, 32, dtype=torch.bfloat16, device=DEV)
    cache = nt.KvCache(k, k.clone())
    q = torch.zeros(2, 4, 32, dtype=torch.bfloat16, device=DEV)
    t, n = i32([[0], [1]]), i32([1, 1])
    with pytest.raises(ValueError):
        nt.ninfer_kv_attention(q[..., :16], cache, t, n)
    with pytest.raises(ValueError):
        nt.ninfer_kv_attention(q, cache, t.long(), n)
    with pytest.raises(ValueError):
        nt.ninfer_kv_attention(q, cache, t, n[:1])
    with pytest.raises(ValueError):
        nt.ninfer_kv_append(cache, q, q, torch.zeros(2, dtype=torch.int64, device=DEV))
    with pytest.raises(ValueError):
        nt.KvCache(k, k[:2])
    with pytest.raises(ValueError):
        nt.KvCache(k.float(), k.float())
    with pytest.raises(nt.NinferError) as e:
        nt.ninfer_kv_attention(q[:, :3], cache, t, n)
    assert e.value.status == 3
    need = nt.ninfer_kv_attention_workspace(cache, 2, 4)
    if need:
        with pytest.raises(nt.NinferError) as e:
            nt.ninfer_kv_attention(q, cache, t, n, workspace=torch.empty(need - 1, dtype=torch.uint8, device=DEV))
        assert e.value.status == 4


def test_c_entry_points_by_ctypes():
    """The C ABI without the binding's checks: one append and one attention through plain ctypes."""
    lib = C.CDLL(nt.LIBRARY_PATH)
    k = torch.zeros(1, 4, 1, 16, dtype=torch.float16, device=DEV)
    v = torch.zeros_like(k)
    c = nt._KvCacheStruct(k.data_ptr(), v.data_ptr(), 1, 4, 1, 16, 64, 16, 16, 1.0, 1.0, nt.F16, 0)
    x = torch.full((1, 1, 16), 2.0, device=DEV)
    slot, u64, vp = torch.tensor([1], device=DEV), C.c_uint64, C.c_void_p
    s = vp(torch.cuda.current_stream().cuda_stream)
    assert lib.ninfer_kv_append(vp(x.data_ptr()), vp(x.data_ptr()), 0, u64(1), u64(16), u64(16), u64(16), u64(16),
                                vp(slot.data_ptr()), C.byref(c), None, s) == 0
    table, length, out = i32([[0]]), i32([2]), torch.zeros(1, 1, 16, device=DEV)
    need = C.c_uint64()
    assert lib.ninfer_kv_attention_workspace(C.byref(c), u64(1), u64(1), C.byref(need)) == 0
    ws = torch.empty(need.value + 256, dtype=torch.uint8, device=DEV)
    assert lib.ninfer_kv_attention(vp(x.data_ptr()), 0, u64(1), u64(1), u64(16), u64(16), C.byref(c), vp(table.data_ptr()), u64(1),
                                   u64(1), vp(length.data_ptr()), C.c_float(0.0), u64(0), vp(out.data_ptr()), 0, None,
                                   vp(ws.data_ptr()), u64(ws.numel()), s) == 0
    torch.cuda.synchronize()
    assert torch.allclose(out, torch.ones_like(out))       # two keys of equal weight, values 0 and 2


@pytest.mark.parametrize("rows", [(1, 1), (1, 4), (2, 8), (4, 9), (9, 8)])
@pytest.mark.parametrize("longest", [130, 520, 1300, 2500, 4000])
@pytest.mark.parametrize("cache,dim", [("bf16", 128), ("f16", 256), ("e4m3", 96)])
def test_attention_few_rows(rows, longest, cache, dim):
    """Few rows of up to a few units a warp: a CTA or a cluster for each, or the line, by the table's width;
    shorter and empty rows among them, which leave CTAs of a cluster without keys."""
    requests, kvh = rows
    rng = np.random.default_rng(longest + dim)
    lengths = ([longest, 1, 0, longest // 2, 33, longest - 1, 17, longest // 3, 5] * 2)[:requests]
    for out in ("bf16", "f32"):
        check_attention(*attention_case(rng, lengths, 3 * kvh, kvh, dim, 16, cache, "bf16", "heads"), out=out,
                        window=0 if out == "bf16" else longest // 2 + 1)
    check_attention(*attention_case(rng, lengths[:2], 12 * kvh, kvh, dim, 16, cache, "f32"), out="f32")


@pytest.mark.parametrize("cache", ["f16", "bf16", "e4m3"])
def test_attention_long_parts_stay_exact(cache):
    """float32 results over 2.6 million keys, 2100 of them in each warp's part, against float64.

    Relative error of the whole result, keys and queries of unit variance, 64 elements: weights 2^-22 from the
    operands' terms and 2^-22 from the exponential, scores about 2^-21 (four cut sums of a score of about one),
    each 16 keys' sum 2^-22 (cut), and their 131 rounded additions 2^-22: 8e-7 in quadrature, 2^-19 allowed. Sums
    that are cut at every one of the additions would be 131 * 2^-25 = 4e-6 off, all towards zero."""
    heads, dim, page, n = 16, 64, 32, 160000
    g = torch.Generator(device="cuda").manual_seed(17)
    dtype = {"f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[cache]
    k, v = (torch.randn(n // page, page, heads, dim, generator=g, device="cuda").to(dtype) for _ in range(2))
    q = torch.randn(1, heads, dim, generator=g, device="cuda")
    table = torch.arange(n // page, dtype=torch.int32, device="cuda").view(1, -1)
    lengths = torch.tensor([n], dtype=torch.int32, device="cuda")
    out = nt.ninfer_kv_attention(q, nt.KvCache(k, v), table, lengths, out_dtype=torch.float32)
    for h in range(heads):
        keys, values = (x[:, :, h].reshape(n, dim).to(torch.float64) for x in (k, v))
        want = torch.softmax(keys @ q[0, h].double() * dim ** -0.5, 0) @ values
        assert (out[0, h].double() - want).norm() <= 2.0 ** -19 * want.norm(), (cache, h)
