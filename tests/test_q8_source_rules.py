"""Rules that the tcgen05 kernels of the 8-bit path keep on their failure paths,
checked on the source text (no GPU needed; a wait that runs out is not provoked).

tcgen05 instructions and barriers marked .aligned are executed by whole warps, and
the lanes of a warp may see a time limit or the abort flag at different times. So

- what a wait returned is agreed on by the warp before the warp acts on it;
- lanes that ran a loop of their own meet again before a barrier of the cluster.

A CTA may leave once the others have read its shared memory. An arrival without
release says nothing about the reads before it, so it has to depend on their values.
"""
import os
import re

from test_source_rules import ROOT, _code

SOURCES = [os.path.join(ROOT, "hybrid_sparse_gemm_b200", "csrc", n) for n in ("q8_split.cu", "q8_wide.cu")]
ACTS = re.compile(r"tmem_ld_\w+\(|issue_slab_i8<|tma_load_\w+\(|load_w\(")


def test_warps_agree_on_what_a_wait_returned():
    seen = 0
    for p in SOURCES:
        code = _code(p)
        for m in re.finditer(r"\bmbar_wait\(|\bmbar_try_wait\(acc_full", code):
            acts = ACTS.search(code, m.end())
            assert acts, p
            line = code.count("\n", 0, m.start()) + 1
            assert "__all_sync(0xffffffffu" in code[m.start() - 40:acts.start()], f"{os.path.basename(p)}:{line}"
            seen += 1
    assert seen >= 7  # producers, issuers and epilogues of both kernels


def test_warps_meet_before_a_cluster_barrier():
    seen = 0
    for p in SOURCES:
        code = _code(p)
        for m in re.finditer(r"\bcluster_sync\(\)|barrier\.cluster\.arrive", code):
            before = code[max(0, m.start() - 120):m.start()]
            assert "__syncwarp()" in before or "__syncthreads()" in before, \
                f"{os.path.basename(p)}:{code.count(chr(10), 0, m.start()) + 1}"
            seen += 1
    assert seen >= 4


def test_an_arrival_that_orders_nothing_depends_on_what_was_read():
    for p in SOURCES:
        code = _code(p)
        for m in re.finditer(r"arrive\.relaxed", code):
            near = code[max(0, m.start() - 400):m.end() + 200]
            assert "@p barrier.cluster.arrive.relaxed" in near and "seen & zero" in near, \
                f"{os.path.basename(p)}:{code.count(chr(10), 0, m.start()) + 1}"
