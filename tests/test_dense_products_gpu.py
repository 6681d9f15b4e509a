"""moe.linear, moe.gated_linear and their gradients against the formulas in 64 bits."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import ACTS, DTYPES, Gate, act_slack, check, half_step, halves, joined, \
    product, randn, slope_slack

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


# (n, R, C): one token, few, past each tile border, ragged everywhere, many
SIZES = [(1, 8, 8), (1, 2880, 2880), (3, 1, 64), (7, 33, 72), (8, 5761, 1408), (31, 40, 2880),
         (32, 256, 512), (33, 257, 520), (64, 2880, 2880), (129, 192, 8), (257, 1000, 1000),
         (300, 77, 2888), (1000, 513, 200), (2048, 2880, 320)]


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("n,R,C", SIZES)
def test_linear(n, R, C, dtype):
    g = gen(n * 7 + R)
    dt = DTYPES[dtype]
    x, w = randn(g, n, C, dtype=dt), randn(g, R, C, dtype=dt, scale=C ** -0.5)
    a, da = product(x, w)
    check(moe.linear(x, w), a, da)
    bias, res = randn(g, R, dtype=dt), randn(g, n, R, dtype=dt)
    b = a + bias.double()
    db = da + 2.0 ** -23 * (a.abs() + bias.double().abs())
    for act, (f, _) in ACTS.items():
        y = f(b)
        slack = act_slack(b, db, act)
        check(moe.linear(x, w, bias=bias, act=act), y, slack, act)
        slack = slack + 2.0 ** -23 * (y.abs() + res.double().abs())
        check(moe.linear(x, w, bias=bias, act=act, residual=res), y + res.double(), slack, act)


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("act", list(ACTS))
@pytest.mark.parametrize("n,R,C", [(1, 8, 8), (5, 64, 72), (32, 264, 512), (33, 512, 1408),
                                   (130, 200, 2888), (513, 1000, 264), (2049, 96, 128),
                                   (4096, 512, 1408)])
def test_linear_backward(n, R, C, act, dtype):
    g = gen(n + R)
    dt = DTYPES[dtype]
    x, w = randn(g, n, C, dtype=dt), randn(g, R, C, dtype=dt, scale=C ** -0.5)
    bias, d_y = randn(g, R, dtype=dt), randn(g, n, R, dtype=dt)
    d_x, d_w, d_bias = moe.linear_backward(d_y, x, w, bias=bias, act=act)
    a, da = product(x, w)
    a, da = a + bias.double(), da + 2.0 ** -22 * (a.abs() + 1)
    d = d_y.double() * ACTS[act][1](a)
    e = torch.zeros_like(d)
    if act != "none":
        e = d_y.double().abs() * slope_slack(a, da, act)
        e = e + (d.abs() + e) * half_step(dt) + torch.finfo(dt).smallest_normal * half_step(dt)
    X, W, D = x.double(), w.double(), d.abs() + e
    check(d_x, d @ W, e @ W.abs() + R * 2.0 ** -23 * (D @ W.abs()), "d_x")
    check(d_w, d.t() @ X, e.t() @ X.abs() + n * 2.0 ** -23 * (D.t() @ X.abs()), "d_w")
    check(d_bias, d.sum(0), e.sum(0) + n * 2.0 ** -23 * D.sum(0), "d_bias")
    got = moe.linear_backward(d_y, x, w, act=act)
    assert got[2] is None


GATED = [(1, 64, 8), (1, 2880, 2880), (3, 72, 40), (8, 512, 1408), (31, 200, 320), (33, 64, 8),
         (64, 2880, 2880), (100, 328, 1000), (257, 512, 136), (1000, 136, 328), (2048, 512, 1408)]


@pytest.mark.parametrize("layout", ["packed", "interleaved"])
@pytest.mark.parametrize("act,par", [("swiglu", {}), ("swiglu", {"limit": 0.7}),
                                     ("swiglu_oai", {}),
                                     ("swiglu_oai", {"alpha": 1.1, "beta": 0.5, "limit": 1.0})])
@pytest.mark.parametrize("n,H,I", GATED)
def test_gated_linear(n, H, I, act, par, layout):
    g = gen(n + I)
    gate = Gate(act, **par)
    params = moe.make_params(act=act, layout=layout, **par)
    for dt in (torch.bfloat16, torch.float16):
        x, w = randn(g, n, H, dtype=dt), randn(g, 2 * I, H, dtype=dt, scale=H ** -0.5)
        a, da = product(x, w)
        (p, u), (dp, du) = halves(a, layout), halves(da, layout)
        h, slack = gate.forward(p, u, dp, du)
        check(moe.gated_linear(x, w, params), h, slack, str(dt))


@pytest.mark.parametrize("dtype", ["bf16", "fp16"])
@pytest.mark.parametrize("layout", ["packed", "interleaved"])
@pytest.mark.parametrize("act,par", [("swiglu", {}), ("swiglu_oai", {"limit": 1.0})])
@pytest.mark.parametrize("n,H,I", [(1, 64, 8), (5, 72, 40), (33, 512, 136), (200, 328, 1000),
                                   (1025, 136, 96), (4096, 512, 1408)])
def test_gated_linear_backward(n, H, I, act, par, layout, dtype):
    g = gen(n + H)
    dt = DTYPES[dtype]
    gate = Gate(act, **par)
    params = moe.make_params(act=act, layout=layout, **par)
    x, w = randn(g, n, H, dtype=dt), randn(g, 2 * I, H, dtype=dt, scale=H ** -0.5)
    d_h = randn(g, n, I, dtype=dt)
    d_x, d_w = moe.gated_linear_backward(d_h, x, w, params)
    a, da = product(x, w)
    (p, u), (dp, du) = halves(a, layout), halves(da, layout)
    d_g, d_u, e_g, e_u = gate.backward(p, u, d_h.double(), dp, du)
    d, e = joined(d_g, d_u, layout), joined(e_g, e_u, layout)
    e = e + (d.abs() + e) * half_step(dt) + torch.finfo(dt).smallest_normal * half_step(dt)
    X, W, D = x.double(), w.double(), d.abs() + e
    check(d_x, d @ W, e @ W.abs() + 2 * I * 2.0 ** -23 * (D @ W.abs()), "d_x")
    check(d_w, d.t() @ X, e.t() @ X.abs() + n * 2.0 ** -23 * (D.t() @ X.abs()), "d_w13")


def test_gradients_against_differences():
    """The gradients of a whole block (gated_linear, linear) along random
    directions against central differences of the formulas in 64 bits."""
    g = gen(11)
    n, H, I = 40, 64, 48
    params = moe.make_params(act="swiglu_oai", layout="interleaved")
    x, w13 = randn(g, n, H), randn(g, 2 * I, H, scale=H ** -0.5)
    w2, bias, d_y = randn(g, H, I, scale=I ** -0.5), randn(g, H), randn(g, n, H)
    h = moe.gated_linear(x, w13, params)
    d_h, d_w2, d_bias = moe.linear_backward(d_y, h, w2, bias=bias, act="silu")
    d_x, d_w13 = moe.gated_linear_backward(d_h, x, w13, params)

    def loss(x, w13, w2, bias):
        p, u = halves(x @ w13.t(), "interleaved")
        hh, _ = Gate("swiglu_oai").forward(p, u, torch.zeros_like(p), torch.zeros_like(u))
        return (d_y.double() * ACTS["silu"][0](hh @ w2.t() + bias)).sum()

    at = [t.double() for t in (x, w13, w2, bias)]
    for i, grad in enumerate((d_x, d_w13, d_w2, d_bias)):
        v = torch.randn(at[i].shape, generator=g, device="cuda", dtype=torch.float64)
        eps = 1e-4
        lo, hi = list(at), list(at)
        lo[i], hi[i] = at[i] - eps * v, at[i] + eps * v
        want = ((loss(*hi) - loss(*lo)) / (2 * eps)).item()
        got = (grad.double() * v).sum().item()
        # each gradient passes at most four roundings to bf16 (h, d, d_h, itself), 2^-8
        # each, of terms that add up along v
        assert abs(got - want) <= 4 * 2.0 ** -8 * (grad.double() * v).abs().sum().item(), i
