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
