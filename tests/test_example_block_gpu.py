"""The dense block of examples/moe_layer.py: it runs, and its gradients are those of
the formula."""
import os
import sys

import pytest
import torch

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                                "examples"))
import moe_layer as example  # noqa: E402

pytestmark = pytest.mark.gpu


def test_runs():
    block, losses, x, residual = example.train_block(H=128, I=160, n=96, steps=3)
    assert len(losses) == 3 and all(v == v for v in losses)
    out = example.serve_mxfp8(block, x, residual)
    assert out.shape == x.shape and torch.isfinite(out).all()


@pytest.mark.parametrize("n", [6, 200])
def test_gradients_against_autograd(n):
    H, I = 256, 320
    block = example.Block(H, I, seed=3)
    g = torch.Generator(device="cuda").manual_seed(4)
    x, residual, d_out = (torch.randn(n, H, generator=g, device="cuda").to(torch.bfloat16)
                          for _ in range(3))
    out, kept = block.forward(x, residual)
    d_x, grads = block.backward(d_out, kept)

    s = (x.double() + residual.double()).requires_grad_()
    leaves = [t.double().requires_grad_() for t in (block.norm, block.w13, block.w2)]
    y = s / torch.sqrt((s * s).mean(1, keepdim=True) + 1e-5) * leaves[0]
    p, u = (y @ leaves[1].t()).chunk(2, dim=1)
    want = (torch.nn.functional.silu(p) * u) @ leaves[2].t() + s
    ref = torch.autograd.grad(want, [s, *leaves], d_out.double())
    # at most six roundings to bf16 lie between the inputs and a gradient (s, y, h,
    # d_h, d, itself), each 2^-8 of its vector's norm at most; random square-ish
    # matrices carry a relative error on without making it larger
    for got, r in zip((out, d_x, *grads), (want, *ref)):
        off = (got.double() - r).norm() / r.norm()
        assert off <= 6 * 2.0 ** -8, off.item()
