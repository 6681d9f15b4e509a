"""examples/moe_layer.py: the layer trained through the library's gradients,
and served with 4-bit experts."""
import os
import sys

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


def test_training_step_against_autograd():
    """Every gradient of the example's step against torch's own for the same
    layer written as dense masked sums in 64 bits (the selection fixed)."""
    import moe_layer as ex
    import mixture_experts_routing_warp_gb300 as moe

    layer = ex.Layer(96, 6, 64, 2, seed=3)
    x = torch.randn(50, 96, device="cuda", generator=torch.Generator("cuda").manual_seed(4))
    d_out = torch.randn(50, 96, device="cuda", generator=torch.Generator("cuda").manual_seed(5))
    out, d_x = ex.forward_backward(layer, x, lambda o: d_out)
    got = [p.grad.clone() for p in layer.parameters()]

    ref = [p.detach().double().requires_grad_() for p in layer.parameters()]
    gate, w13, w2 = ref
    xx = x.double().requires_grad_()
    indx, _ = moe.route((x @ layer.gate.t()).detach(), 2)
    logits = xx @ gate.t()
    w = torch.softmax(torch.gather(logits, 1, indx.long()), 1)
    full = torch.zeros(50, 6, dtype=torch.float64, device="cuda").scatter(1, indx.long(), w)
    a = torch.einsum("th,eih->tei", xx, w13)
    h = torch.nn.functional.silu(a[..., :64]) * a[..., 64:]
    want = (full[..., None] * torch.einsum("tei,ehi->teh", h, w2)).sum(1)
    want.backward(d_out.double())
    # the gate weights are bf16 in the layer (half a step, 2^-9 of each here
    # below 1); everything else is fp32 (torch's products at most 2^-10 of a
    # sum's magnitude where they run on reduced-precision units)
    tol = 2.0 ** -8 + 2.0 ** -10
    for name, a_, b_ in (("out", out, want), ("gate", got[0], gate.grad), ("w13", got[1], w13.grad),
                         ("w2", got[2], w2.grad)):
        rel = (a_.double() - b_).norm() / b_.norm()
        assert rel <= tol, (name, rel.item())
    # d_x is the experts' share (the router's reaches x through logits)
    a = torch.einsum("th,eih->tei", xx, w13)
    h = torch.nn.functional.silu(a[..., :64]) * a[..., 64:]
    y = (full.detach()[..., None] * torch.einsum("tei,ehi->teh", h, w2)).sum(1)
    share = torch.autograd.grad(y, xx, d_out.double())[0]
    assert (d_x.double() - share).norm() <= tol * share.norm()


def test_training_learns():
    import moe_layer as ex

    losses = ex.train(H=128, E=4, I=64, k=2, n=256, steps=40)
    assert losses[-1] < 0.7 * losses[0], losses


@pytest.mark.parametrize("H,E,I,k", [(256, 8, 192, 2), (2880, 4, 2880, 4)])
def test_decode_with_4_bit_experts(H, E, I, k):
    """forward_q4 against moe.forward on the weights that the codes stand for,
    which bf16 holds exactly: what differs is moe.forward's rounding of h and
    of each slot's output to bf16 (2^-9 each, independent) and the final
    rounding of both (2^-9 each)."""
    import moe_layer as ex

    got, want = ex.decode(H=H, E=E, I=I, k=k, tokens=5)
    rel = (got.double() - want.double()).norm() / want.double().norm()
    assert rel <= 4 * 2.0 ** -9, rel.item()
