"""Products of MXFP8 operands, and MXFP8 outputs, against the formulas in 64 bits."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import ACTS, Gate, act_slack, check, check_mx8, halves, mx8_rows, mx8_value, \
    product, randn

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


@pytest.mark.parametrize("n,R,C", [(1, 8, 32), (5, 33, 96), (8, 2880, 2880), (33, 200, 128),
                                   (1, 2880, 2880), (9, 77, 1440), (16, 5761, 2880), (17, 96, 160),
                                   (64, 5761, 1408), (129, 193, 160), (257, 1000, 2880),
                                   (1000, 513, 512), (2047, 5760, 2880)])
def test_linear(n, R, C):
    g = gen(n + R)
    (xc, xs), (wc, ws) = mx8_rows(g, n, C), mx8_rows(g, R, C, C ** -0.5)
    x, w = moe.Mx8(xc, xs), moe.Mx8(wc, ws)
    a, da = product(mx8_value(xc, xs), mx8_value(wc, ws))
    check(moe.linear(x, w), a, da)
    for dt in (torch.bfloat16, torch.float16):
        bias, res = randn(g, R, dtype=dt), randn(g, n, R, dtype=dt)
        b = a + bias.double()
        db = da + 2.0 ** -23 * (a.abs() + bias.double().abs())
        for act, (f, _) in ACTS.items():
            y = f(b)
            slack = act_slack(b, db, act) + 2.0 ** -23 * (y.abs() + res.double().abs())
            got = moe.linear(x, w, bias=bias, act=act, residual=res, dtype=dt)
            check(got, y + res.double(), slack, act)


@pytest.mark.parametrize("layout", ["packed", "interleaved"])
@pytest.mark.parametrize("act", ["swiglu", "swiglu_oai"])
@pytest.mark.parametrize("n,H,I", [(1, 32, 32), (7, 96, 40), (8, 2880, 2880), (16, 1440, 416),
                                   (17, 64, 96), (40, 160, 64),
                                   (129, 512, 1408), (600, 288, 352), (2048, 2880, 96)])
def test_gated_linear(n, H, I, act, layout):
    g = gen(n + I)
    (xc, xs), (wc, ws) = mx8_rows(g, n, H), mx8_rows(g, 2 * I, H, H ** -0.5)
    x, w = moe.Mx8(xc, xs), moe.Mx8(wc, ws)
    params = moe.make_params(act=act, layout=layout)
    a, da = product(mx8_value(xc, xs), mx8_value(wc, ws))
    (p, u), (dp, du) = halves(a, layout), halves(da, layout)
    h, slack = Gate(act).forward(p, u, dp, du)
    check(moe.gated_linear(x, w, params), h, slack)
    check(moe.gated_linear(x, w, params, dtype=torch.float16), h, slack)
    if I % 32 == 0:
        q = moe.gated_linear(x, w, params, mx8=True)
        check_mx8(q.codes, q.scales, h, slack)


@pytest.mark.parametrize("layout", ["packed", "interleaved"])
@pytest.mark.parametrize("n,H,I", [(1, 64, 32), (8, 2880, 2880), (13, 264, 160), (33, 72, 96), (257, 512, 1408),
                                   (1500, 328, 160)])
def test_gated_linear_writes_mx8(n, H, I, layout):
    """16-bit operands, the result in 8 bits."""
    g = gen(n + I)
    x, w = randn(g, n, H), randn(g, 2 * I, H, scale=H ** -0.5)
    a, da = product(x, w)
    (p, u), (dp, du) = halves(a, layout), halves(da, layout)
    h, slack = Gate("swiglu").forward(p, u, dp, du)
    q = moe.gated_linear(x, w, moe.make_params(act="swiglu", layout=layout), mx8=True)
    check_mx8(q.codes, q.scales, h, slack)


@pytest.mark.parametrize("n", [140, 5, 16])
def test_every_scale_and_code(n):
    """Each row's own scales and each code at its place: x and w have one group
    that is not zero, with a scale of its own; all 254 finite codes occur."""
    C, R = 288, 256
    codes = torch.arange(256, dtype=torch.uint8, device="cuda")
    codes[127] = codes[255] = 0                       # the two NaNs
    wc = torch.zeros(R, C, dtype=torch.uint8, device="cuda")
    for j in range(C // 32):
        wc[j::C // 32, 32 * j] = codes[j::C // 32]
    ws = (100 + torch.arange(R * C // 32, device="cuda") % 50).to(torch.uint8).view(R, C // 32)
    xc = torch.full((n, C), 56, dtype=torch.uint8, device="cuda")   # 1.0
    xs = (110 + torch.arange(n * C // 32, device="cuda") % 37).to(torch.uint8).view(n, C // 32)
    wc, xc = wc.view(torch.float8_e4m3fn), xc.view(torch.float8_e4m3fn)
    want = mx8_value(xc, xs) @ mx8_value(wc, ws).t()
    got = moe.linear(moe.Mx8(xc, xs), moe.Mx8(wc, ws))
    assert torch.equal(got.double(), want)            # one product each: exact in bf16


@pytest.mark.parametrize("n", [200, 18, 16, 6])
def test_nan_reaches_its_rows_alone(n):
    g = gen(1)
    R, C = 224, 192
    (xc, xs), (wc, ws) = mx8_rows(g, n, C), mx8_rows(g, R, C)
    want, _ = product(mx8_value(xc, xs), mx8_value(wc, ws))
    xs[n - 2, 3] = 255                                   # a scale that is NaN
    wc.view(torch.uint8)[150, 100] = 127              # a code that is NaN
    got = moe.linear(moe.Mx8(xc, xs), moe.Mx8(wc, ws))
    bad = torch.zeros(n, R, dtype=torch.bool, device="cuda")
    bad[n - 2], bad[:, 150] = True, True
    assert torch.equal(torch.isnan(got), bad)
    assert torch.allclose(got.double()[~bad], want[~bad], rtol=2.0 ** -7, atol=1e-3)


@pytest.mark.parametrize("n", [300, 1, 11])
def test_block_in_8_bits(n):
    """norm -> gated_linear -> linear, 8 bits between them, as a served block
    runs; each step against the formula on the rows that it was given."""
    g = gen(2)
    H, I = 320, 416
    x, res = randn(g, n, H), randn(g, n, H)
    w = (1 + 0.1 * randn(g, H, dtype=torch.float32)).to(torch.bfloat16)
    (c13, s13), (c2, s2) = mx8_rows(g, 2 * I, H, H ** -0.5), mx8_rows(g, H, I, I ** -0.5)
    params = moe.make_params(act="swiglu_oai", layout="interleaved")
    y, s = moe.rms_norm(x, w, 1e-5, residual=res, mx8=True)
    h = moe.gated_linear(y, moe.Mx8(c13, s13), params, mx8=True)
    out = moe.linear(h, moe.Mx8(c2, s2), residual=s)
    a, da = product(mx8_value(y.codes, y.scales), mx8_value(c13, s13))
    want, slack = Gate("swiglu_oai").forward(a[:, ::2], a[:, 1::2], da[:, ::2], da[:, 1::2])
    check_mx8(h.codes, h.scales, want, slack)
    a, da = product(mx8_value(h.codes, h.scales), mx8_value(c2, s2))
    check(out, a + s.double(), da + 2.0 ** -23 * (a.abs() + s.double().abs()))
