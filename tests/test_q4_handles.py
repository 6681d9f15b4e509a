"""The handle of 4-bit weights: what it shows is what the calls read, for as long as it lives."""
import pytest

import mixture_experts_routing_warp_gb300 as moe


@pytest.mark.parametrize("name", ["codes", "scales", "matrix_scale", "fmt"])
def test_a_handle_takes_no_other_tensors(name):
    w = moe.Q4Weight.__new__(moe.Q4Weight)
    with pytest.raises(AttributeError):
        setattr(w, name, None)
