"""Decode-step operators, the part that needs no GPU: hand-worked values of the
oracle, and the refusals, which come back before any device work (fake aligned
addresses stand in for device buffers)."""
import ctypes as C

import numpy as np
import pytest

import bit_gemv_gb300 as nt
from oracle import decode as od

OK, INVALID, SHAPE, SIZE, ALIGN, OVERFLOW = 0, 1, 3, 4, 5, 8
FAKE = 1 << 20
lib = nt._lib


# ----------------------------------------------------------------- oracle ---
def test_oracle_rounding_by_hand():
    # e4m3 around 1: steps of 1/8, ties to even; the subnormal step is 2^-9; saturation at 448
    x = [1.0, 1.0625, 1.1875, 1.07, 2.0 ** -10, 3 * 2.0 ** -10, 460.0, 1e9, -1e9, 464.0]
    assert od.round_to(x, "e4m3", True).tolist() == [1.0, 1.0, 1.25, 1.125, 0.0, 2.0 ** -8, 448.0, 448.0, -448.0, 448.0]
    assert od.round_to([1 + 2.0 ** -8, 1 + 3 * 2.0 ** -8], "bf16").tolist() == [1.0, 1 + 2.0 ** -6]
    assert od.round_to([65520.0, 65519.9, 2.0 ** -25], "f16").tolist() == [np.inf, 65504.0, 0.0]
    r = np.random.default_rng(0).standard_normal(1000) * 10.0 ** np.random.default_rng(1).integers(-9, 5, 1000)
    assert np.array_equal(od.round_to(r, "f16"), r.astype(np.float16).astype(np.float64))
    assert np.array_equal(od.round_to(r, "f32"), r.astype(np.float32).astype(np.float64))


def test_oracle_tables_by_hand():
    # pages of 4: request 0 holds 5 tokens (pages 7, 2) and gets 4 more (one fresh page), request 1 nothing, 2 starts with 5
    table = [[7, 2, -1], [-1, -1, -1], [-1, -1, -1]]
    t, slots, pos, rows, off, lens, counts, status = od.kv_tables([5, 0, 0], [4, 0, 5], 4, [9, 4, 1], table, 11)
    assert t.tolist() == [[7, 2, 9], [-1, -1, -1], [4, 1, -1]]
    assert slots.tolist() == [9, 10, 11, 36, 16, 17, 18, 19, 4, -1, -1]
    assert pos.tolist() == [5, 6, 7, 8, 0, 1, 2, 3, 4, -1, -1] and rows.tolist() == [0] * 4 + [2] * 5 + [-1] * 2
    assert off.tolist() == [0, 4, 4, 9] and lens.tolist() == [9, 0, 5] and counts.tolist() == [9, 3] and status == 0
    # a short list, a short row and too few slots
    t, slots, *_, counts, status = od.kv_tables([0], [13], 4, [3], [[-1, -1]], 6)
    assert t.tolist() == [[3, -1]] and slots.tolist() == [12, 13, 14, 15, -1, -1] and counts.tolist() == [13, 4] and status == 7


def test_oracle_attention_by_hand():
    # two keys at right angles: scores ln 3 and 0, weights 3/4 and 1/4; the window of 1 leaves the second
    k = np.zeros((2, 1, 1, 2))
    k[1, 0, 0], k[0, 0, 0] = [1, 0], [0, 1]
    v = np.zeros_like(k)
    v[1, 0, 0], v[0, 0, 0] = [4, 0], [0, 8]
    q = np.array([[[np.log(3), 0.0]]])
    out, lse, _, _ = od.kv_attention(q, k, v, np.array([[1, 0]]), [2], 1.0)
    assert np.allclose(out[0, 0], [3, 2]) and np.isclose(lse[0, 0], np.log(4))
    assert np.allclose(od.kv_attention(q, k, v, np.array([[1, 0]]), [2], 1.0, window=1)[0][0, 0], [0, 8])
    out, lse, _, _ = od.kv_attention(q, k, v, np.array([[1, 0]]), [0], 1.0)
    assert not out.any() and lse[0, 0] == -np.inf


def test_oracle_logits_by_hand():
    x = [[2.0, -2.0, 1.0, 0.0]]
    y = od.logits_process(x, np.array([[0, 1, 1, 0, 9]]), [5], [1], [2.0], [0.5], [0.25], [{2: 4.0, 1: 1.0}],
                          np.array([[True, True, True, False]]))
    # 0: 2/2 - 0.25 - 0.5, 1: -2*2 - 0.5 - 0.5 + 1, 2: 1 + 4, 3 forbidden
    assert y.tolist() == [[0.25, -4.0, 5.0, -np.inf]]


# --------------------------------------------------------------- refusals ---
def cache(**kw):
    c = dict(k=FAKE, v=FAKE, pages=8, page_size=16, kv_heads=2, head_dim=64, page_stride=2048, token_stride=128,
             head_stride=64, k_scale=1.0, v_scale=1.0, dtype=nt.BF16, reserved=0)
    c.update(kw)
    return nt._KvCacheStruct(*[c[f] for f, _ in nt._KvCacheStruct._fields_])


BAD_CACHES = [(dict(k=None), INVALID), (dict(v=None), INVALID), (dict(dtype=nt.F32), INVALID), (dict(dtype=7), INVALID),
              (dict(k_scale=0.0), INVALID), (dict(v_scale=float("inf")), INVALID), (dict(k_scale=float("nan")), INVALID),
              (dict(k_scale=-1.0), INVALID), (dict(reserved=1), INVALID), (dict(pages=0), SHAPE), (dict(page_size=0), SHAPE),
              (dict(kv_heads=0), SHAPE), (dict(pages=2 ** 31), SHAPE), (dict(head_dim=0), SHAPE), (dict(head_dim=264), SHAPE),
              (dict(head_dim=60), SHAPE), (dict(head_dim=72, dtype=nt.E4M3), SHAPE), (dict(token_stride=100), ALIGN),
              (dict(page_stride=2052), ALIGN), (dict(head_stride=60), ALIGN), (dict(k=FAKE + 8), ALIGN),
              (dict(v=FAKE + 2), ALIGN), (dict(page_stride=2 ** 40), OVERFLOW), (dict(token_stride=2 ** 24), OVERFLOW)]


@pytest.mark.parametrize("bad,status", BAD_CACHES)
def test_cache_refusals(bad, status):
    c, b = cache(**bad), C.c_uint64()
    assert lib.ninfer_kv_attention_workspace(C.byref(c), 1, 2, C.byref(b)) == status
    assert lib.ninfer_kv_append(FAKE, FAKE, nt.BF16, 4, 128, 64, 128, 64, FAKE, C.byref(c), None, None) == status


def test_append_refusals():
    def append(k=FAKE, v=FAKE, dt=nt.BF16, n=4, ks=128, kh=64, vs=128, vh=64, slots=FAKE, status=None):
        return lib.ninfer_kv_append(k, v, dt, n, ks, kh, vs, vh, slots, C.byref(cache()), status, None)
    assert append(k=None) == INVALID and append(v=None) == INVALID and append(slots=None) == INVALID
    assert append(dt=nt.E4M3) == INVALID
    assert append(n=0) == SHAPE and append(n=2 ** 31) == SHAPE
    assert append(k=FAKE + 4) == ALIGN and append(slots=FAKE + 4) == ALIGN and append(status=FAKE + 2) == ALIGN
    assert append(ks=132) == ALIGN and append(vh=60) == ALIGN and append(dt=nt.F32, ks=130) == ALIGN
    assert lib.ninfer_kv_append(FAKE, FAKE, nt.BF16, 4, 128, 64, 128, 64, FAKE, None, None, None) == INVALID


def test_attention_refusals():
    ws = C.c_uint64()
    assert lib.ninfer_kv_attention_workspace(C.byref(cache()), 0, 2, C.byref(ws)) == SHAPE
    assert lib.ninfer_kv_attention_workspace(C.byref(cache()), 1, 3, C.byref(ws)) == SHAPE
    assert lib.ninfer_kv_attention_workspace(C.byref(cache()), 2 ** 30, 64, C.byref(ws)) == OVERFLOW
    assert lib.ninfer_kv_attention_workspace(C.byref(cache()), 1, 2, None) == INVALID

    def attend(q=FAKE, qd=nt.BF16, n=2, heads=4, qr=256, qh=64, table=FAKE, width=3, stride=3, lengths=FAKE, scale=0.125,
               window=0, out=FAKE, od_=nt.BF16, lse=None, wsp=FAKE, wsb=1 << 40):
        return lib.ninfer_kv_attention(q, qd, n, heads, qr, qh, C.byref(cache()), table, width, stride, lengths, scale,
                                       window, out, od_, lse, wsp, wsb, None)
    for name in ("q", "table", "lengths", "out"):
        assert attend(**{name: None}) == INVALID, name
    assert attend(qd=nt.E4M3) == INVALID and attend(od_=9) == INVALID
    assert attend(scale=float("nan")) == INVALID and attend(scale=float("inf")) == INVALID
    assert attend(n=0) == SHAPE and attend(heads=0) == SHAPE and attend(heads=3) == SHAPE
    assert attend(width=0) == SHAPE and attend(stride=2) == SHAPE and attend(width=2 ** 30, stride=2 ** 30) == OVERFLOW
    assert attend(q=FAKE + 2) == ALIGN and attend(qr=252) == ALIGN and attend(qh=36) == ALIGN and attend(out=FAKE + 8) == ALIGN
    assert attend(table=FAKE + 2) == ALIGN and attend(lengths=FAKE + 1) == ALIGN and attend(lse=FAKE + 2) == ALIGN
    assert b"attention" in lib.ninfer_last_error()


def test_tables_refusals():
    def tables(lengths=FAKE, new=None, n=4, page=16, free=FAKE, count=9, table=FAKE, width=5, stride=5, slots=FAKE, pos=FAKE,
               rows=FAKE, cap=8, off=FAKE, lo=FAKE, counts=FAKE, status=None):
        return lib.ninfer_kv_tables(lengths, new, n, page, free, count, table, width, stride, slots, pos, rows, cap, off, lo,
                                    counts, status, None)
    assert tables(lengths=None) == INVALID and tables(table=None) == INVALID and tables(free=None) == INVALID
    assert tables(n=0) == SHAPE and tables(page=0) == SHAPE and tables(width=0, stride=0) == SHAPE and tables(stride=4) == SHAPE
    assert tables(cap=2 ** 31) == SHAPE and tables(count=2 ** 31) == SHAPE and tables(page=2 ** 31) == SHAPE
    assert tables(slots=FAKE + 4) == ALIGN and tables(lengths=FAKE + 2) == ALIGN and tables(counts=FAKE + 1) == ALIGN


def test_logits_refusals():
    def process(x=FAKE, xs=100, out=2 * FAKE, os_=100, dt=nt.F32, rows=2, vocab=100, status=None, **kw):
        c = nt._LogitsControls(**kw)
        return lib.ninfer_logits_process(x, xs, out, os_, dt, rows, vocab, C.byref(c), status, None)
    assert process(x=None) == INVALID and process(out=None) == INVALID and process(dt=nt.E4M3) == INVALID
    assert lib.ninfer_logits_process(FAKE, 4, FAKE, 4, 0, 1, 4, None, None, None) == INVALID
    assert process(history=FAKE, history_stride=5) == INVALID
    assert process(bias_ids=FAKE) == INVALID and process(bias_ids=FAKE, bias_values=FAKE) == INVALID
    assert process(rows=0) == SHAPE and process(vocab=0) == SHAPE and process(xs=99) == SHAPE and process(os_=99) == SHAPE
    assert process(out=FAKE, os_=104) == SHAPE
    assert process(mask=FAKE, mask_row_count=1, mask_stride=4) == SHAPE
    assert process(mask=FAKE, mask_row_count=2, mask_stride=3) == SHAPE
    assert process(mask=FAKE, mask_row_count=0, mask_stride=4, mask_rows=FAKE) == SHAPE
    assert process(x=FAKE + 4) == ALIGN and process(presence=FAKE + 2) == ALIGN and process(status=FAKE + 1) == ALIGN


def test_binding_refuses_host_tensors():
    torch = pytest.importorskip("torch")
    k = torch.zeros(2, 4, 1, 16, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        nt.KvCache(k, k)
    with pytest.raises(ValueError):
        nt.ninfer_logits_process(torch.zeros(1, 5))
    with pytest.raises(ValueError):
        nt.ninfer_kv_tables(torch.zeros(1, dtype=torch.int32), None, 4, None, torch.zeros(1, 2, dtype=torch.int32), 1)
