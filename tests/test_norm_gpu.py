"""moe.rms_norm and its gradients against the formulas in 64 bits."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import DTYPES, check, check_mx8, half_step, randn

pytestmark = pytest.mark.gpu
EPS = 1e-5
STEP = 2.0 ** -24  # a rounding in fp32


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def sum_slack(H):
    """Relative error of a sum of H terms of one sign in fp32 and of 1 / rms."""
    return (min(H, 256) + 40) * STEP  # at most 8 vectors of 8 (or a loop of 128) per thread


# one element, odd lengths, past each number of threads and vectors, rows read twice
LENGTHS = [1, 2, 8, 31, 32, 64, 100, 255, 1001, 1408, 2048, 2880, 2879, 4099, 8192, 16392, 40000,
           65536]


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", LENGTHS)
def test_norm(H, dtype):
    dt = DTYPES[dtype]
    for n in (1, 5, 400 if H < 5000 else 7):
        g = gen(H + n)
        x = randn(g, n, H, dtype=dt) * torch.exp(randn(g, n, 1, dtype=torch.float32)).to(dt)
        res = randn(g, n, H, dtype=dt)
        for wt in (dt, torch.float32, None):
            w = None if wt is None else (1 + 0.3 * randn(g, H, dtype=torch.float32)).to(wt)
            y = moe.rms_norm(x, w, EPS)
            z, s = moe.rms_norm(x, w, EPS, residual=res)
            total = x.double() + res.double()
            # the sum: one fp32 rounding, then the type's
            check(s, total, total.abs() * STEP, "sum")
            for got, v in ((y, x.double()), (z, s.double())):
                want = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
                want = want if w is None else want * w.double()
                check(got, want, want.abs() * (sum_slack(H) + 4 * STEP), "y")


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", [32, 64, 96, 1408, 2880, 4128, 33024])
def test_norm_mx8(H, dtype):
    dt = DTYPES[dtype]
    for n in (1, 6, 333 if H < 5000 else 5):
        g = gen(H + n)
        x, res = randn(g, n, H, dtype=dt), randn(g, n, H, dtype=dt)
        w = (1 + 0.3 * randn(g, H, dtype=torch.float32)).to(dt)
        y = moe.rms_norm(x, w, EPS, mx8=True)
        z, s = moe.rms_norm(x, w, EPS, residual=res, mx8=True)
        for got, v in ((y, x.double()), (z, s.double())):
            want = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS) * w.double()
            check_mx8(got.codes, got.scales, want, want.abs() * (sum_slack(H) + 4 * STEP))


@pytest.mark.parametrize("dtype", list(DTYPES))
@pytest.mark.parametrize("H", LENGTHS)
def test_norm_backward(H, dtype):
    dt = DTYPES[dtype]
    for n in (1, 5, 3000 if H < 3000 else 9):
        g = gen(H + n)
        x, d_y, d_sum = (randn(g, n, H, dtype=dt) for _ in range(3))
        for wt in (dt, torch.float32):
            w = (1 + 0.3 * randn(g, H, dtype=torch.float32)).to(wt)
            X, D, W = x.double(), d_y.double(), w.double()
            r = 1 / torch.sqrt((X * X).mean(1, keepdim=True) + EPS)
            v, dw = X * r, D * W
            m = (dw * v).mean(1, keepdim=True)
            d_x = r * (dw - v * m)
            rel = sum_slack(H) + 8 * STEP
            slack = r * rel * (dw.abs() + v.abs() * (dw * v).abs().mean(1, keepdim=True) * 3)
            got, d_w = moe.rms_norm_backward(d_y, x, w, EPS)
            check(got, d_x, slack, "d_x")
            # a column: at most n terms in a row, in any order
            check(d_w, (D * v).sum(0), (D * v).abs().sum(0) * (rel + n * STEP), "d_weight")
            got, _ = moe.rms_norm_backward(d_y, x, w, EPS, d_sum=d_sum)
            check(got, d_x + d_sum.double(),
                  slack + STEP * (d_x.abs() + d_sum.double().abs()), "d_x + d_sum")
        got, none = moe.rms_norm_backward(d_y, x, None, EPS)
        assert none is None
        m = (D * v).mean(1, keepdim=True)
        check(got, r * (D - v * m),
              r * rel * (D.abs() + v.abs() * (D * v).abs().mean(1, keepdim=True) * 3), "no weight")


@pytest.mark.parametrize("dtype", list(DTYPES))
def test_rows_at_any_alignment(dtype):
    """Bases and rows off 16 bytes, between guard values."""
    dt = DTYPES[dtype]
    g = gen(3)
    for H in (64, 77, 2880):
        for off in (1, 3):
            n = 6
            buf = randn(g, n * H + off, dtype=dt)
            x = buf[off:].view(n, H)
            out = torch.full((n * H + off + 8,), 7.0, dtype=dt, device="cuda")
            y = moe.rms_norm(x, None, EPS, out=out[off:off + n * H].view(n, H))
            v = x.double()
            want = v / torch.sqrt((v * v).mean(1, keepdim=True) + EPS)
            check(y, want, want.abs() * (sum_slack(H) + 4 * STEP))
            assert (out[:off] == 7).all() and (out[off + n * H:] == 7).all()


def test_values_that_are_not_finite():
    x = torch.randn(4, 64, device="cuda")
    x[1, 3] = float("nan")
    x[2, 40] = float("inf")
    x[3] = 0
    y = moe.rms_norm(x, None, EPS)
    assert torch.isfinite(y[0]).all() and torch.isnan(y[1]).all() and (y[3] == 0).all()
    assert torch.isnan(y[2, 40]) and (y[2, :40] == 0).all()   # x / inf
    q = moe.rms_norm(x, None, EPS, mx8=True)
    assert (q.scales[1] == 255).all()
    assert q.scales[2, 1] == 255 and q.scales[2, 0] == 0 and (q.codes[2, :32].float() == 0).all()
    assert (q.scales[3] == 0).all() and (q.codes[3].float() == 0).all()


def test_gradient_against_differences():
    g = gen(5)
    x, d_y = torch.randn(6, 40, device="cuda"), torch.randn(6, 40, device="cuda")
    w = torch.rand(40, device="cuda") + 0.5
    d_x, d_w = moe.rms_norm_backward(d_y, x, w, EPS)

    def loss(x, w):
        return (d_y.double() * x / torch.sqrt((x * x).mean(1, keepdim=True) + EPS) * w).sum()

    for grad, at in ((d_x, 0), (d_w, 1)):
        p = [x.double(), w.double()]
        v = torch.randn(p[at].shape, generator=g, device="cuda", dtype=torch.float64)
        lo, hi = list(p), list(p)
        lo[at], hi[at] = p[at] - 1e-5 * v, p[at] + 1e-5 * v
        want = (loss(*hi) - loss(*lo)) / 2e-5
        got = (grad.double() * v).sum()
        # fp32 sums of at most 40 terms; the differences are good to 1e-8
        assert abs(got - want) <= 1e-5 * (grad.double() * v).abs().sum()
