"""The row handles of 8-bit rows: a call reads the tensors that the handle shows, where they
lie at that call."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import mx8_rows


def test_a_handle_takes_no_other_tensors():
    """Without a GPU: codes and scales are read-only."""
    for name in ("codes", "scales"):
        assert getattr(moe.Mx8, name).fset is None
        with pytest.raises(AttributeError):
            setattr(moe.Mx8.__new__(moe.Mx8), name, torch.zeros(1))


@pytest.mark.gpu
def test_memory_that_moves_behind_the_handle():
    g = torch.Generator(device="cuda").manual_seed(1)
    (xc, xs), (wc, ws), (vc, vs) = (mx8_rows(g, r, 64) for r in (40, 96, 96))
    x, w = moe.Mx8(xc, xs), moe.Mx8(wc, ws)
    first, want = moe.linear(x, w), moe.linear(x, moe.Mx8(vc, vs))
    assert not torch.equal(first, want)
    with pytest.raises(AttributeError):
        w.codes = vc
    wc.data, ws.data = vc, vs                     # other memory for the same tensors
    assert torch.equal(moe.linear(x, w), want)
    out = moe.Mx8(torch.empty(40, 64, dtype=torch.float8_e4m3fn, device="cuda"),
                  torch.empty(40, 2, dtype=torch.uint8, device="cuda"))
    rows = torch.randn(40, 64, generator=g, device="cuda")
    q = moe.rms_norm(rows, None, mx8=True)
    moved = torch.zeros_like(out.codes)
    out.codes.data = moved
    moe.rms_norm(rows, None, mx8=True, out=out)
    assert torch.equal(moved.view(torch.uint8), q.codes.view(torch.uint8))


@pytest.mark.gpu
@pytest.mark.parametrize("which", ["codes", "scales"])
def test_memory_of_another_shape_is_refused(which):
    g = torch.Generator(device="cuda").manual_seed(2)
    (xc, xs), (wc, ws) = mx8_rows(g, 40, 64), mx8_rows(g, 96, 64)
    x, w = moe.Mx8(xc, xs), moe.Mx8(wc, ws)
    t = wc if which == "codes" else ws
    t.data = t[:8].clone()                        # fewer rows than the handle's
    with pytest.raises(ValueError, match="no longer"):
        moe.linear(x, w)
    t.data = torch.zeros(t.shape[1], 96, dtype=t.dtype, device="cuda").t()
    with pytest.raises(ValueError, match="no longer"):
        moe.linear(x, w)
