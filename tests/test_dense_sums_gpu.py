"""Long sums of the dense blocks: gradients of weights over 2^18 rows and more, products of 65536
features, and gradients along random directions. Compared as whole arrays, relative
to their norm: an element-wise bound of so many roundings is wider than the sums themselves.

Of the norm of a result: its rounding takes at most eps / 2; an operand that was rounded
before, eps / 2 (its elements are off independently); an accumulator of fp32 that takes 16
products at a time 2^-23 per addition, all of one sign."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import ACTS, Gate, halves, joined, mx8_rows, mx8_value, randn

pytestmark = pytest.mark.gpu
HALF = 2.0 ** -8                                   # half a step of bf16, relative


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def off(got, want):
    return ((got.double() - want).norm() / want.norm()).item()


@pytest.fixture
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    yield
    torch.cuda.empty_cache()


def test_gated_weight_gradient_of_many_rows(room):
    """d of more than 2^31 elements, every row of it random."""
    g, I, H = gen(1), 4096, 64
    n = (1 << 31) // (2 * I) + 300
    x, d_h = randn(g, n, H), randn(g, n, I)
    w13 = randn(g, 2 * I, H, scale=0.125)
    d_x, d_w = moe.gated_linear_backward(d_h, x, w13, moe.make_params(act="swiglu", layout="packed"))
    gate, W, want, worst = Gate("swiglu"), w13.double(), 0, 0.0
    for lo in range(0, n, 1 << 14):
        X, D = x[lo:lo + (1 << 14)].double(), d_h[lo:lo + (1 << 14)].double()
        p, u = halves(X @ W.t(), "packed")
        zero = torch.zeros_like(p)
        d = joined(*gate.backward(p, u, D, zero, zero)[:2], "packed")
        want = want + d.t() @ X
        worst = max(worst, off(d_x[lo:lo + (1 << 14)], d @ W))
    assert off(d_w, want) <= 2 * HALF + n / 16 * 2.0 ** -23
    assert worst <= 2 * HALF + 2 * I / 16 * 2.0 ** -23


def test_linear_weight_gradient_of_many_rows(room):
    g, R, C = gen(2), 4096, 40
    n = (1 << 31) // R + 77
    x, d_y = randn(g, n, C), randn(g, n, R)
    d_x, d_w, d_bias = moe.linear_backward(d_y, x, randn(g, R, C), bias=randn(g, R))
    want, column = 0, 0
    for lo in range(0, n, 1 << 14):
        X, D = x[lo:lo + (1 << 14)].double(), d_y[lo:lo + (1 << 14)].double()
        want, column = want + D.t() @ X, column + D.sum(0)
    assert off(d_w, want) <= HALF + n / 16 * 2.0 ** -23
    assert off(d_bias, column) <= HALF + n * 2.0 ** -24


@pytest.mark.parametrize("H", [8192, 8191])
def test_norm_weight_gradient_of_many_rows(room, H):
    g, n = gen(H), (1 << 31) // H + 300
    x, d = randn(g, n, H), randn(g, n, H)
    _, d_w = moe.rms_norm_backward(d, x, torch.rand(H, device="cuda") + 0.5, 1e-5)
    want = 0
    for lo in range(0, n, 1 << 13):
        X, D = x[lo:lo + (1 << 13)].double(), d[lo:lo + (1 << 13)].double()
        want = want + (D * X / torch.sqrt((X * X).mean(1, keepdim=True) + 1e-5)).sum(0)
    # a thread adds at most n / 304 rows, 304 sums are joined; 1 / rms to 2^-20
    assert off(d_w, want) <= (n / 304 + 304) * 2.0 ** -24 + 2.0 ** -20


@pytest.mark.parametrize("n", [1, 20, 40, 300])
def test_65536_features(n):
    g, C = gen(n), 65536
    x, w = randn(g, n, C), randn(g, 96, C, scale=C ** -0.5)
    long = C / 16 * 2.0 ** -23
    assert off(moe.linear(x, w), x.double() @ w.double().t()) <= HALF + long
    h = moe.gated_linear(x, w, moe.make_params(act="swiglu", layout="interleaved"))
    p, u = halves(x.double() @ w.double().t(), "interleaved")
    # silu's slope is at most 1.1
    assert off(h, torch.nn.functional.silu(p) * u) <= HALF + 4 * long
    (xc, xs), (wc, ws) = mx8_rows(g, n, C), mx8_rows(g, 96, C, C ** -0.5)
    got = moe.linear(moe.Mx8(xc, xs), moe.Mx8(wc, ws))
    assert off(got, mx8_value(xc, xs) @ mx8_value(wc, ws).t()) <= HALF + long
    # as the features that a gradient sums over
    d_y, x, w = randn(g, n, C), randn(g, n, 64), randn(g, C, 64, scale=0.125)
    d_x, d_w, _ = moe.linear_backward(d_y, x, w)
    assert off(d_x, d_y.double() @ w.double()) <= HALF + long
    assert off(d_w, d_y.double().t() @ x.double()) <= HALF + long


@pytest.mark.parametrize("act,layout", [("swiglu_oai", "interleaved"), ("swiglu", "packed")])
@pytest.mark.parametrize("n", [6, 40])
def test_gradients_along_directions(n, act, layout):
    """A block's gradients along 16 random directions against central differences in 64 bits:
    an error e of a gradient shows as a normal deviate of size |e|, so over 16 directions its mean
    square is that of |e| within a factor of 4."""
    g = gen(n)
    H, I, steps = 64, 48, 1e-4
    params = moe.make_params(act=act, layout=layout)
    x, w13 = randn(g, n, H), randn(g, 2 * I, H, scale=H ** -0.5)
    w2, bias, d_y = randn(g, H, I, scale=I ** -0.5), randn(g, H), randn(g, n, H)
    h = moe.gated_linear(x, w13, params)
    d_h, d_w2, d_bias = moe.linear_backward(d_y, h, w2, bias=bias, act="gelu")
    d_x, d_w13 = moe.gated_linear_backward(d_h, x, w13, params)

    def loss(x, w13, w2, bias):
        p, u = halves(x @ w13.t(), layout)
        hh, _ = Gate(act).forward(p, u, torch.zeros_like(p), torch.zeros_like(u))
        return (d_y.double() * ACTS["gelu"][0](hh @ w2.t() + bias)).sum()

    at = [t.double() for t in (x, w13, w2, bias)]
    for i, grad in enumerate((d_x, d_w13, d_w2, d_bias)):
        grad, square = grad.double(), 0.0
        for _ in range(16):
            v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
            lo, hi = list(at), list(at)
            lo[i], hi[i] = at[i] - steps * v, at[i] + steps * v
            diff = (loss(*hi) - loss(*lo)) / (2 * steps) - (grad * v).sum()
            square += diff.item() ** 2 / 16
        # at most five roundings to bf16 on the way to a gradient (h, d, d_h, d, itself), and
        # the factor of 4 in the square
        assert square ** 0.5 <= 2 * 5 * HALF * grad.norm().item(), i
