"""A thread whose bounded wait gave up waits at the end for the cluster's other threads to leave.  If a
block-wide barrier followed, they would wait for it there and it for them, for ever.  That can only be
shown by a lost copy or total, so the order is held in the source."""
import os
import re

import pytest

SOURCE = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "bit_linear_gb300", "csrc", "scan.cu")
BARRIER = re.compile(r"__syncthreads|sync_cuts|bar(rier)?\.sync|cluster_wait|cluster_sync")
LEAVE = re.compile(r"\b(cluster_leave|leave_late)\b")


def _kernels():
    """(name, body) of every kernel that joins a cluster."""
    text = re.sub(r"//[^\n]*", "", open(SOURCE).read())
    for m in re.finditer(r"__global__[^;{]*?\b(tern_\w+)\s*\([^;{]*\)\s*\{", text):
        depth, at = 1, m.end()
        while depth:
            depth += {"{": 1, "}": -1}.get(text[at], 0)
            at += 1
        body = text[m.end():at]
        if "open_exchange" in body:
            yield m.group(1), body


@pytest.mark.parametrize("name,body", list(_kernels()), ids=[k for k, _ in _kernels()])
def test_nothing_waits_for_a_thread_that_leaves_late(name, body):
    first = LEAVE.search(body)
    assert first, "a wait that gave up has to let the peers leave first"
    assert not BARRIER.search(body[first.start():]), name


def test_both_kernels_are_looked_at():
    assert sorted(k for k, _ in _kernels()) == ["tern_scan_bwd_kernel", "tern_scan_fwd_kernel"]
