"""Decode-step operators where results or memory are easily lost, the part that needs no
GPU: the oracle at such inputs, and calls that are refused before any device work (fake aligned
addresses stand in for device buffers)."""
import ctypes as C

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
