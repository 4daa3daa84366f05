"""csrc/overlap.h against all bytes written out, and the layer operators' refusals of outputs that share memory with what else a call reads
or writes. (The calls are all refused: fake addresses stand in for device buffers.)"""
import os
import random
import shutil
import subprocess

import pytest

import bit_gemv_gb300 as nt
from test_layer_host import FAKE, INVALID, delta, norm, rotary, sample

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemv_gb300", "csrc")
PROGRAM = r"""
#include <cstdio>
#include "overlap.h"
int main() {
    unsigned long long a[6], b[6];
    while (scanf("%llu %llu %llu %llu %llu %llu %llu %llu %llu %llu %llu %llu", a, a + 1, a + 2, a + 3, a + 4, a + 5, b, b + 1, b + 2, b + 3, b + 4, b + 5) == 12) {
        const ninfer::Span x((void *)a[0], a[1], a[2], a[3], a[4], a[5]), y((void *)b[0], b[1], b[2], b[3], b[4], b[5]);
        printf("%d %d\n", x.meets(y), y.meets(x));
    }
}
"""


def bytes_of(at, run, rows, row, parts, part):
    return {at + i * (row if rows > 1 else 0) + j * (part if parts > 1 else 0) + b for i in range(rows) for j in range(parts) for b in range(run)}


@pytest.mark.skipif(not shutil.which("g++"), reason="no g++")
def test_spans_meet_where_bytes_are_shared(tmp_path):
    (tmp_path / "m.cpp").write_text(PROGRAM)
    subprocess.run(["g++", "-O1", "-std=c++17", "-fsanitize=undefined", "-fno-sanitize-recover", "-I", CSRC, "-o", str(tmp_path / "m"), str(tmp_path / "m.cpp")], check=True)
    rng = random.Random(1)
    cases = []
    for _ in range(6000):
        shared = rng.choice([0, 7, 12, 24])         # often one stride for both, as of views of one buffer
        spans = [(rng.randint(100, 180), rng.randint(1, 9), rng.randint(1, 5), shared or rng.randint(0, 30), rng.randint(1, 4), rng.choice([0, 3, 4, 8, 13, 40]))
                 for _ in range(2)]
        cases.append(spans)
    cases.append([(2 ** 62, 2 ** 40, 2 ** 20, 2 ** 41, 1, 0), (2 ** 62 + 2 ** 40, 2 ** 40, 2 ** 20, 2 ** 41, 1, 0)])
    told = subprocess.run([str(tmp_path / "m")], input="\n".join(" ".join(map(str, a + b)) for a, b in cases), capture_output=True, text=True, check=True).stdout.split("\n")
    assert told[len(cases) - 1] == "0 0"
    met = 0
    for (a, b), line in zip(cases[:-1], told):
        want = int(bool(bytes_of(*a) & bytes_of(*b)))
        assert line == f"{want} {want}", (a, b)
        met += want
    assert 1000 < met < 5000


# x 4 rows of 64 bf16 (128 bytes a row), heads of q 64 bf16, ...
@pytest.mark.parametrize("kw", [
    dict(out=FAKE + 16), dict(out=FAKE - 16), dict(out=FAKE + 3 * 128), dict(out=FAKE * 2 + 256), dict(out=FAKE * 3 - 2, group=32), dict(out=FAKE * 4 + 64),
    dict(sum=FAKE * 2 + 128), dict(sum=FAKE * 6 + 256), dict(sum=FAKE * 4), dict(sum=FAKE + 128), dict(out=FAKE * 5 - 128),
    dict(x_stride=128, out_stride=128, out=FAKE + 64, rows=2), dict(x_stride=128, out_stride=96, out=FAKE + 128)])
def test_norm_refuses_outputs_that_overlap(kw):
    assert norm(**kw) == INVALID


BASE = dict(positions=FAKE * 10, frequencies=FAKE * 11, q_weight=FAKE * 12, k_weight=FAKE * 13)


@pytest.mark.parametrize("kw", [
    dict(q_out=FAKE + 128), dict(q_out=FAKE - 512), dict(k_out=2 * FAKE + 128), dict(q_out=2 * FAKE + 16), dict(k_out=FAKE + 1024), dict(q_out=2 * FAKE - 512),
    dict(q_out=4 * FAKE, k_out=4 * FAKE), dict(q_out=4 * FAKE, k_out=4 * FAKE + 1024), dict(q_out=FAKE * 10 - 1024), dict(q_out=FAKE * 11), dict(q_out=FAKE * 12),
    dict(k_out=FAKE * 13 + 16), dict(q_out_token=512, q_token=512, q_out=FAKE + 1024),
    # heads of 64 in rows of [q, gate] pairs, the keys behind them reaching into the last gate's place
    dict(q_head=128, q_out_head=128, q_token=1024, q_out_token=1024, k=FAKE + 2 * 3 * 128, k_out=FAKE + 2 * 3 * 128, k_token=1024, k_out_token=1024),
    # outputs whose own heads or tokens share memory
    dict(q_out=4 * FAKE, q_out_head=32), dict(q_out=4 * FAKE, q_out_head=0), dict(k_out=5 * FAKE, k_out_token=0), dict(k_out=5 * FAKE, k_out_token=64)])
def test_rotary_refuses_outputs_that_overlap(kw):
    assert rotary(**{**BASE, **kw}) == INVALID


NAMES = ("q", "k", "v", "log_decay", "beta", "state", "state_slots", "offsets", "lengths", "out", "status")
APART = {n: FAKE * 16 * (i + 1) for i, n in enumerate(NAMES)}
SPACE = dict(workspace=FAKE * 1024, bytes_=2 ** 24)


@pytest.mark.parametrize("kw", [
    *[dict(out=APART[n]) for n in NAMES if n not in ("out", "v")], *[dict(out=APART[n] - 16) for n in NAMES if n != "out"],
    *[dict(status=APART[n]) for n in NAMES if n != "status"], *[{n: APART["state"] + 4 * 8192 * 4} for n in NAMES if n != "state"],
    *[{n: FAKE * 1024 + 256} for n in NAMES],
    dict(out=APART["v"], out_dtype=nt.F32), dict(out=APART["v"], out_dtype=nt.F16), dict(out=APART["v"], v_token=256),
    dict(out=APART["state"] + 32768 * 4, slot_stride=32768), dict(out=APART["state"] + 32832 * 4 - 2288, slot_stride=32832)])
def test_gated_delta_refuses_outputs_that_overlap(kw):
    assert delta(**{**SPACE, **APART, **kw}) == INVALID


@pytest.mark.parametrize("name", [n for n in NAMES if n not in ("offsets", "out", "v")])
def test_gated_delta_of_single_tokens_refuses_outputs_that_overlap(name):
    assert delta(None, 0, **{**APART, "offsets": 0, "tokens": 3, "out": APART[name]}) == INVALID


@pytest.mark.parametrize("kw", [dict(tokens=FAKE), dict(tokens=FAKE + 300 * 4 - 4), dict(logprobs=FAKE * 2 + 8), dict(logprobs=FAKE * 7 + 8), dict(logprobs=FAKE * 7),
                                dict(logprobs=FAKE + 400), dict(tokens=FAKE * 8 - 8), dict(tokens=FAKE * 5 + 4), dict(tokens=FAKE * 6 - 8)])
def test_sample_refuses_outputs_that_overlap(kw):
    names = ("logits", "temperature", "top_p", "min_p", "top_k", "random", "tokens", "logprobs")
    assert sample(**{**{n: FAKE * (i + 1) for i, n in enumerate(names)}, **kw}) == INVALID
