"""A block's barriers are reached by all of its threads in one place: none of them is the
body of a condition on a thread's own share of the work."""
import glob
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                    "mixture_experts_routing_warp_gb300", "csrc")


@pytest.mark.parametrize("path", sorted(glob.glob(os.path.join(CSRC, "*.cu*"))), ids=os.path.basename)
def test_no_barrier_under_a_condition_of_its_own(path):
    text = re.sub(r"//[^\n]*|/\*.*?\*/", "", open(path).read(), flags=re.S)
    found = re.findall(r"(?:\bif\s*\([^;{}]*\)|\belse)\s*__syncthreads\s*\(\s*\)", text)
    assert not found, found


def test_a_warp_leaves_a_bounded_wait_together():
    """The dense products' roles are whole warps (votes, exchanges and TMEM loads of all lanes
    follow): whether a wait gave up is put to the vote before any lane acts on it."""
    text = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, "dense_gemm.cu")).read())
    waits = [m.start() for m in re.finditer(r"\bwait_bounded\s*\(", text)]
    assert waits
    for at in waits:
        statements = text[at:].split(";")
        assert "__all_sync(0xffffffffu, ok)" in statements[1], text[at:at + 200]
