"""GELU and its gradient far below zero, where (1 + erf) / 2 is a small number that a sum with 1
would round away: relative to the value, in every kernel that applies them."""
import math

import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import DTYPES, check

pytestmark = pytest.mark.gpu

# few rows, tiles, rows off 16 bytes, a sum in parts
SIZES = [(4, 64, 64), (40, 64, 64), (300, 61, 64), (200, 256, 8192)]


def rows(n, R, C, dtype):
    """Arguments from -12 to 1 as products with one term each: exact."""
    x = torch.zeros(n, C, device="cuda")
    x[:, :R] = torch.linspace(-12.0, 1.0, n * R, device="cuda").view(n, R)
    w = torch.zeros(R, C, dtype=dtype, device="cuda")
    w[torch.arange(R), torch.arange(R)] = 1.0
    x = x.to(dtype)
    return x, w, x[:, :R].double()


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,R,C", SIZES)
def test_values(n, R, C, dtype):
    dt = DTYPES[dtype]
    x, w, v = rows(n, R, C, dt)
    want = 0.5 * v * torch.special.erfc(-v / math.sqrt(2))
    # erfc(u) moves by 2 u du / u relative to itself for large u: u^2 <= 72, its argument
    # is off by 1.5 * 2^-24, the function by 4 * 2^-23, two products by 2^-24 each
    check(moe.linear(x, w, act="gelu"), want, want.abs() * (2 * 72 * 1.5 + 8 + 2 + 8) * 2.0 ** -24)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,R,C", [(4, 64, 64), (40, 64, 64), (200, 256, 8192)])
def test_slopes(n, R, C, dtype):
    dt = DTYPES[dtype]
    x, w, v = rows(n, R, C, dt)
    d_x, _, _ = moe.linear_backward(torch.ones(n, R, dtype=dt, device="cuda"), x, w, act="gelu")
    below = 0.5 * torch.special.erfc(-v / math.sqrt(2))
    pdf = torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    # the first term as above; the second: exp's argument (72 at most, three roundings), the
    # function itself 2 + 1.2 * 72 steps of 2^-23, products; the sum
    slack = below * (2 * 72 * 1.5 + 18) * 2.0 ** -24 + \
        v.abs() * pdf * (72 * 3 + 2 * 89 + 8) * 2.0 ** -24
    got = d_x[:, :R]
    # d is rounded once to its type, and one product with 1 keeps it; exp flushes below 2^-126
    check(got, below + v * pdf, slack + 12 * 2.0 ** -126)
    assert (d_x[:, R:] == 0).all()
