"""Kernels whose CTAs write into one another's shared memory: the CTAs of a cluster run together, but nothing says that
they have all started, and shared memory of a CTA that has not must not be touched. So a barrier of the cluster, or
its two halves, stands before the first such write. (The order is read in the source: a GPU whose CTAs happen to
start together shows nothing.)"""
import os
import re

import pytest

from deterministic_token_logprob_gb300.build import CSRC

WRITE = re.compile(r"\bst_cluster_\w+\(|\bmbar_arrive_cluster\(")
STARTED = re.compile(r"\bcluster_wait\(\)|\bcluster_sync\(\)")


def body(file, head):
    """The text of the function whose definition `head` starts, without comments."""
    with open(os.path.join(CSRC, file)) as f:
        s = re.sub(r"//[^\n]*", "", f.read())
    at = s.index("{", s.index(head))
    depth = 0
    for i in range(at, len(s)):
        depth += {"{": 1, "}": -1}.get(s[i], 0)
        if depth == 0:
            return s[at:i]
    raise AssertionError(head)


@pytest.mark.parametrize("file,head,write", [
    ("rlk_embedding.cu", "void sort_tokens(", WRITE),
    ("rlk_logits_row.cuh", "void row_pass(", re.compile(r"\bleaf_pass<")),
    ("rlk_distill.cu", "void __launch_bounds__(STEP_THREADS, STEP_CTAS) distill_step_kernel(", re.compile(r"\bleaf_pass<")),
])
def test_every_cta_has_started(file, head, write):
    s = body(file, head)
    first, started = write.search(s), STARTED.search(s)
    assert first and started and started.start() < first.start()
    if started.group().startswith("cluster_wait"):
        arrive = s.index("cluster_arrive()")
        assert arrive < started.start() and "cluster_wait" not in s[:arrive]


def test_halves_of_the_sorts_barrier_pair_up():
    """Each thread arrives once, before the passes, and waits once, in the first: both where there are other CTAs, which
    all threads see alike."""
    s = body("rlk_embedding.cu", "void sort_tokens(")
    assert s.count("cluster_arrive()") == s.count("cluster_wait()") == 1
    assert s.index("cluster_arrive()") < s.index("for (int pass = 0;")
    assert re.search(r"\n  if \(ctas > 1\) cluster_arrive\(\);", s)
    assert re.search(r"\n    if \(pass == 0 && ctas > 1\) cluster_wait\(\);", s)


def test_no_other_source_writes_across_ctas():
    """Another kernel that does belongs into the list above."""
    writers = set()
    for f in sorted(os.listdir(CSRC)):
        with open(os.path.join(CSRC, f)) as g:
            s = re.sub(r"//[^\n]*", "", g.read())
        if re.search(r"st\.\w+\.cluster\.shared::cluster|st_cluster_\w+\(", s):
            writers.add(f)
    assert writers == {"rlk_embedding.cu", "rlk_logits_row.cuh", "rlk_gemm.cuh", "rlk_ptx.cuh"}
