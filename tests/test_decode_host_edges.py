"""Decode-step operators where results or memory are easily lost, the part that needs no
GPU: the oracle at such inputs, and calls that are refused before any device work (fake aligned
addresses stand in for device buffers)."""
import copy
import ctypes as C

import pytest

import bit_gemv_gb300 as nt
from oracle import decode as od

OK, INVALID, SHAPE = 0, 1, 3
FAKE = 1 << 20
lib = nt._lib


def test_oracle_reports_rows_too_short_for_tokens_in_held_pages():
    # 40 tokens need three pages of 16 and so does the 41st; the row has two, and no page is taken
    _, slots, *_, counts, status = od.kv_tables([40], [1], 16, [5, 6], [[1, 2]], 1)
    assert slots.tolist() == [-1] and counts.tolist() == [1, 0] and status == 2
    assert od.kv_tables([40], [0], 16, [5, 6], [[1, 2]], 1)[-1] == 0        # no new token: nothing is lost
    assert od.kv_tables([31], [1], 16, [5, 6], [[1, 2]], 1)[-1] == 0


def logits(x=FAKE, out=2 * FAKE, rows=2, vocab=100, stride=100, **kw):
    return lib.ninfer_logits_process(x, stride, out, stride, nt.F32, rows, vocab, C.byref(nt._LogitsControls(**kw)), None, None)


def test_logits_histories_are_shorter_than_a_table_entry_counts():
    # an entry counts to 2^30 - 1; within 9216 of 2^31 the kernel's index would pass 31 bits
    for stride in (2 ** 30, 2 ** 31 - 9000, 2 ** 31 - 1):
        assert logits(history=FAKE, history_lengths=FAKE, history_stride=stride) == SHAPE
    assert b"history_stride" in lib.ninfer_last_error()


def tables(lengths=FAKE, new=2 * FAKE, n=4, free=3 * FAKE, count=9, table=4 * FAKE, width=5, stride=8, slots=5 * FAKE, pos=6 * FAKE,
           rows=7 * FAKE, cap=8, off=8 * FAKE, lo=9 * FAKE, counts=10 * FAKE, status=11 * FAKE):
    return lib.ninfer_kv_tables(lengths, new, n, 16, free, count, table, width, stride, slots, pos, rows, cap, off, lo, counts,
                                status, None)


def test_tables_outputs_that_overlap_inputs():
    # lengths_out = lengths is what a loop would write: CTAs that come later would count from the new lengths
    assert tables(lo=FAKE) == INVALID
    assert b"lengths_out may not be lengths" in lib.ninfer_last_error()
    assert tables(lo=FAKE + 12) == INVALID and tables(lo=FAKE - 12) == INVALID
    assert tables(lo=2 * FAKE) == INVALID and tables(off=FAKE - 16) == INVALID and tables(slots=3 * FAKE + 32) == INVALID
    assert tables(pos=FAKE - 28) == INVALID and tables(rows=2 * FAKE + 8) == INVALID
    assert tables(counts=3 * FAKE + 32) == INVALID and tables(status=2 * FAKE + 12) == INVALID
    # rows of 20 bytes, 32 apart
    assert tables(table=FAKE) == INVALID and tables(table=3 * FAKE - 96) == INVALID
    assert tables(counts=4 * FAKE + 32 + 16) == INVALID and tables(counts=4 * FAKE + 3 * 32 - 4) == INVALID
    assert tables(slots=4 * FAKE + 24) == INVALID and tables(status=4 * FAKE + 3 * 32 + 16) == INVALID


# ---------------------------------------------------------------- binding ---
class Tensor:
    """What the binding asks of a contiguous CUDA tensor."""
    is_cuda = True

    def __init__(self, at, dtype, *shape, device=0):
        self.at, self.dtype, self.shape, self.index = at, dtype, shape, device

    def data_ptr(self):
        return self.at

    def numel(self):
        n = 1
        for s in self.shape:
            n *= s
        return n

    def stride(self):
        strides = [1]
        for s in self.shape[:0:-1]:
            strides.insert(0, strides[0] * s)
        return tuple(strides)

    def is_contiguous(self):
        return True

    def get_device(self):
        return self.index

    @property
    def device(self):
        return "cuda:%d" % self.index

    def detach(self):
        return copy.copy(self)


def buffers(device=0, requests=3, capacity=5):
    torch = pytest.importorskip("torch")
    i32 = lambda at, n: Tensor(at * FAKE, torch.int32, n, device=device)  # noqa: E731
    return nt.KvTables(Tensor(FAKE, torch.int32, requests, 4, device=device), Tensor(2 * FAKE, torch.int64, capacity, device=device),
                       i32(3, capacity), i32(4, capacity), i32(5, requests + 1), i32(6, requests), i32(7, 2))


def test_kv_tables_looks_at_its_buffers_again():
    nt._types()
    t = buffers()
    _, table, tokens, requests, *_ = t._addresses(5, 0)
    assert table == (FAKE, 3, 4, 4) and tokens == (2 * FAKE, 3 * FAKE, 4 * FAKE) and requests == (5 * FAKE, 6 * FAKE, 7 * FAKE)
    t.positions.at = 30 * FAKE                              # memory replaced in place, as by resize_ or set_
    t.lengths.at = 60 * FAKE
    _, _, tokens, requests, *_ = t._addresses(5, 0)
    assert tokens == (2 * FAKE, 30 * FAKE, 4 * FAKE) and requests == (5 * FAKE, 60 * FAKE, 7 * FAKE)
    t.block_table.shape = (3, 9)                            # longer rows at the same place
    assert t._addresses(5, 0)[1] == (FAKE, 3, 9, 9)
    t.block_table.at = 10 * FAKE
    assert t._addresses(5, 0)[1] == (10 * FAKE, 3, 9, 9)
    t.slots.at, t.slots.shape = 20 * FAKE, (4,)
    for _ in range(2):
        with pytest.raises(ValueError):
            t._addresses(5, 0)


def test_kv_tables_copies_have_buffers_of_their_own():
    nt._types()
    t = buffers()
    t._addresses(5, 0)
    other = copy.deepcopy(t)
    for x in other:
        x.at += FAKE // 2
    assert other._addresses(5, 0)[2] == tuple(a + FAKE // 2 for a in t._addresses(5, 0)[2])


def test_kv_cache_looks_at_its_pools_again():
    torch = pytest.importorskip("torch")
    k, v = (Tensor(at * FAKE, torch.bfloat16, 8, 16, 2, 64) for at in (1, 2))
    c = nt.KvCache(k, v, 0.5, 0.25)
    k.at, v.at = 3 * FAKE, 4 * FAKE
    for t in (k, v):
        t.shape = (32, 16, 2, 64)
    s = c._current(0)._obj
    assert (s.k, s.v, s.pages, s.page_stride, s.k_scale, s.v_scale) == (3 * FAKE, 4 * FAKE, 32, 2048, 0.5, 0.25) and c.pages == 32
    k.at, k.shape = 5 * FAKE, (16, 16, 2, 64)               # one pool alone
    with pytest.raises(ValueError):
        c._current(0)


def test_arguments_on_different_devices_are_refused(monkeypatch):
    """Before the library is asked: it would read one GPU's memory from another."""
    torch = pytest.importorskip("torch")
    nt._types()
    bf16, i32, i64 = torch.bfloat16, torch.int32, torch.int64
    monkeypatch.setattr(nt, "_several", False)

    def pools(k=0, v=0):
        return Tensor(FAKE, bf16, 8, 16, 2, 64, device=k), Tensor(2 * FAKE, bf16, 8, 16, 2, 64, device=v)
    with pytest.raises(ValueError):
        nt.KvCache(*pools(0, 1))
    for cache, first, others in ((1, 0, [0] * 4), (0, 0, [1, 0, 0, 0]), (0, 0, [0, 1, 0, 0]), (0, 0, [0, 0, 1, 0]), (0, 0, [0, 0, 0, 1])):
        c = nt.KvCache(*pools(cache, cache))
        with pytest.raises(ValueError):
            nt.ninfer_kv_attention(Tensor(3 * FAKE, bf16, 3, 4, 64, device=first), c, Tensor(4 * FAKE, i32, 3, 2, device=others[0]),
                                   Tensor(5 * FAKE, i32, 3, device=others[1]), out=Tensor(6 * FAKE, bf16, 3, 4, 64, device=others[2]),
                                   workspace=Tensor(7 * FAKE, torch.uint8, 1 << 30, device=others[3]))
        if others[2] == others[3] == 0:
            with pytest.raises(ValueError):
                nt.ninfer_kv_append(c, Tensor(3 * FAKE, bf16, 3, 2, 64, device=first), Tensor(4 * FAKE, bf16, 3, 2, 64, device=others[0]),
                                    Tensor(5 * FAKE, i64, 3, device=others[1]))
    lengths, free = Tensor(12 * FAKE, i32, 3), Tensor(13 * FAKE, i32, 7)
    for out, fr, table in ((buffers(1), free, None), (buffers(), Tensor(FAKE, i32, 7, device=1), None),
                           (buffers(), free, Tensor(FAKE, i32, 3, 4, device=1))):
        with pytest.raises(ValueError):
            nt.ninfer_kv_tables(lengths, None, 16, fr, table or out.block_table, 5, out=out)
    x = Tensor(FAKE, torch.float32, 2, 100)
    for kw in (dict(out=Tensor(2 * FAKE, torch.float32, 2, 100, device=1)), dict(repetition=Tensor(2 * FAKE, torch.float32, 2, device=1)),
               dict(mask=Tensor(2 * FAKE, i32, 2, 4, device=1))):
        with pytest.raises(ValueError):
            nt.ninfer_logits_process(x, **dict(dict(out=Tensor(3 * FAKE, torch.float32, 2, 100)), **kw))
    # where there are several, the current one is the one that the library launches on
    monkeypatch.setattr(nt, "_several", True)
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 1)
    with pytest.raises(ValueError):
        nt.KvCache(*pools())
    nt.KvCache(*pools(1, 1))
