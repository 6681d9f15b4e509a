"""Matrices of more than 2^31 elements: the last rows of the results against the
formulas, where an offset that passes 32 bits would show."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import Gate, check, check_mx8, halves, half_step, joined, mx8_rows, mx8_value, \
    product

pytestmark = pytest.mark.gpu
STEP = 2.0 ** -24


@pytest.fixture(autouse=True)
def room():
    free, _ = torch.cuda.mem_get_info()
    if free < 60 << 30:
        pytest.skip("needs 60 GB")
    yield
    torch.cuda.empty_cache()


def rows(n, cols, last, seed):
    """bf16 rows, random in the last `last` and in the first, 1 elsewhere."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.ones(n, cols, dtype=torch.bfloat16, device="cuda")
    for part in (x[:last], x[n - last:]):
        part.copy_(torch.randn(part.shape, generator=g, device="cuda"))
    return x


@pytest.mark.parametrize("H", [8192, 8191])
def test_norm(H):
    n, k = (1 << 31) // H + 300, 40
    x, d = rows(n, H, k, 1), rows(n, H, k, 2)
    w = torch.rand(H, device="cuda") + 0.5
    y = moe.rms_norm(x, w, 1e-5)
    d_x, d_w = moe.rms_norm_backward(d, x, w, 1e-5)
    for s in (slice(0, k), slice(n - k, n)):
        X, D = x[s].double(), d[s].double()
        r = 1 / torch.sqrt((X * X).mean(1, keepdim=True) + 1e-5)
        v, dw = X * r, D * w.double()
        check(y[s], v * w.double(), (v * w.double()).abs() * 300 * STEP)
        want = r * (dw - v * (dw * v).mean(1, keepdim=True))
        check(d_x[s], want, r * 310 * STEP * (dw.abs() + 3 * v.abs() *
                                              (dw * v).abs().mean(1, keepdim=True)))
    if H % 32 == 0:
        q = moe.rms_norm(x, w, 1e-5, mx8=True)
        v = x[n - k:].double()
        want = v / torch.sqrt((v * v).mean(1, keepdim=True) + 1e-5) * w.double()
        check_mx8(q.codes[n - k:], q.scales[n - k:], want, want.abs() * 300 * STEP)


@pytest.mark.parametrize("R", [8192, 8191])
def test_linear(R):
    n, C, k = (1 << 31) // R + 300, 64, 300
    x = rows(n, C, k, 3)
    w = torch.randn(R, C, device="cuda").mul_(0.125).to(torch.bfloat16)
    res = rows(n, R, k, 4)
    y = moe.linear(x, w, residual=res)
    for s in (slice(0, k), slice(n - k, n)):
        a, da = product(x[s], w)
        a = a + res[s].double()
        check(y[s], a, da + 2.0 ** -23 * (a.abs() + res[s].double().abs()))


def test_gradients():
    """The contraction over 2^18 rows and more, d of more than 2^31 elements."""
    I, H, k = 4096, 64, 300
    n = (1 << 31) // (2 * I) + 300
    x, d_h = rows(n, H, k, 5), rows(n, I, k, 6)
    w13 = torch.randn(2 * I, H, device="cuda").mul_(0.125).to(torch.bfloat16)
    params = moe.make_params(act="swiglu", layout="packed")
    h = moe.gated_linear(x, w13, params)
    d_x, d_w = moe.gated_linear_backward(d_h, x, w13, params)
    gate = Gate("swiglu")
    for s in (slice(0, k), slice(n - k, n)):
        a, da = product(x[s], w13)
        (p, u), (dp, du) = halves(a, "packed"), halves(da, "packed")
        want, slack = gate.forward(p, u, dp, du)
        check(h[s], want, slack)
        d_g, d_u, e_g, e_u = gate.backward(p, u, d_h[s].double(), dp, du)
        d, e = joined(d_g, d_u, "packed"), joined(e_g, e_u, "packed")
        e = e + (d.abs() + e) * half_step(torch.bfloat16) + 2.0 ** -126
        W = w13.double()
        check(d_x[s], d @ W, e @ W.abs() + 2 * I * 2.0 ** -23 * ((d.abs() + e) @ W.abs()))
    assert torch.isfinite(d_w).all()


def test_mx8():
    I, H, k = 4096, 64, 300
    n = (1 << 31) // I + 300
    g = torch.Generator(device="cuda").manual_seed(7)
    codes = torch.full((n, H), 56, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    scales = torch.full((n, H // 32), 127, dtype=torch.uint8, device="cuda")
    c, s = mx8_rows(g, k, H)
    codes.view(torch.uint8)[n - k:] = c.view(torch.uint8)
    scales[n - k:] = s
    wc, ws = mx8_rows(g, 2 * I, H, 0.125)
    params = moe.make_params(act="swiglu_oai", layout="interleaved")
    q = moe.gated_linear(moe.Mx8(codes, scales), moe.Mx8(wc, ws), params, mx8=True)
    a, da = product(mx8_value(c, s), mx8_value(wc, ws))
    (p, u), (dp, du) = halves(a, "interleaved"), halves(da, "interleaved")
    h, slack = Gate("swiglu_oai").forward(p, u, dp, du)
    check_mx8(q.codes[n - k:], q.scales[n - k:], h, slack)
