"""Shared memory of another CTA of a cluster may be touched only once that CTA has begun: in every kernel that does so, in the
order of its source, each CTA arrives at the cluster's barrier and waits there before the first
access. Read from the source, because a late CTA cannot be had at will on a GPU."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_gemv_gb300", "csrc")
ARRIVE = re.compile(r"cluster_arrive\(\)|barrier\.cluster\.arrive(?:\.relaxed|\.release)?\.aligned;\" |cluster_sync\(\)|join\(\)")
WAIT = re.compile(r"cluster_wait\(\)|barrier\.cluster\.wait(?:\.acquire)?\.aligned;\" |cluster_sync\(\)|join\(\)")
# file, kernel, its calls that reach another CTA's shared memory
KERNELS = [("sample.cu", "sample_kernel", r"row\.(?:cluster_max|exchange|merge|template merge|list|adopt|locate)"),
           ("gemv_ptq1_int.cu", "gemv_ptq1_int_kernel", r"mapa_shared|st_cluster"),
           ("gemv_pq2_int.cu", "gemv_pq2_int_kernel", r"rotate_pack2")]


def body(name, kernel):
    """The kernel's source without comments, from its name to the brace that closes it."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    at = re.search(r"__global__[^{;]*?\b" + kernel + r"\([^{;]*\{", text, re.S).end()
    depth, end = 1, at
    while depth:
        depth += {"{": 1, "}": -1}.get(text[end], 0)
        end += 1
    return text[at:end]


def condition(text, at):
    """The condition of the statement at a place: on its line, or that of the block that it begins."""
    return re.findall(r"if \(([^(){}]*)\)\s*(?:\{[^{}]*)?$", text[max(at - 200, 0):at].replace("asm volatile(\"", "").rstrip())


@pytest.mark.parametrize("name,kernel,remote", KERNELS)
def test_no_access_before_every_cta_has_begun(name, kernel, remote):
    text = body(name, kernel)
    arrive, wait, first = ARRIVE.search(text), WAIT.search(text), re.search(remote, text)
    assert arrive and wait and first
    assert arrive.start() <= wait.start() < first.start()
    # a wait without an arrival before it, or the reverse, has no meaning
    assert condition(text, arrive.start()) == condition(text, wait.start())


def test_every_file_with_such_accesses_is_listed():
    found = {f for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh")) and f != "async.cuh" and "mapa_shared(" in open(os.path.join(CSRC, f)).read()}
    # attention's kernel joins through cluster_sync alone
    assert found == {n for n, _, _ in KERNELS} | {"kv_attention.cuh"}
