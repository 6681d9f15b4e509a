"""moe.route_backward on logits and gradients that are not finite: the formula
d_e = p_e (up_e - sum p up) decides, term by term."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")


def setup(E, k=4, n=9, seed=1):
    g = torch.Generator(device="cuda").manual_seed(seed)
    z = torch.randn(n, E, generator=g, device="cuda")
    indx = torch.argsort(torch.rand(n, E, generator=g, device="cuda"), 1)[:, :k].int().contiguous()
    return z, indx, torch.randn(n, k, generator=g, device="cuda")


@pytest.mark.parametrize("E", [8, 37, 128, 255, 256])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_logit_that_is_not_finite_over_all(E, value):
    z, indx, d = setup(E)
    clean = moe.route_backward(z, indx, d, "softmax_all")
    for e in (0, E // 2, int(indx[4, 1])):
        bad = z.clone()
        bad[4, e] = value
        got = moe.route_backward(bad, indx, d, "softmax_all")
        assert got[4].isnan().all()
        got[4] = clean[4]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("E", [8, 37, 128])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_logit_that_is_not_finite_over_the_selected(E, value):
    """A selected one makes the selected gradients NaN and leaves the others
    zero; one that is not selected takes no part."""
    z, indx, d = setup(E)
    clean = moe.route_backward(z, indx, d, "softmax_topk")
    chosen = torch.zeros(E, dtype=torch.bool, device="cuda")
    chosen[indx[4].long()] = True
    for e in range(0, E, max(1, E // 8)):
        bad = z.clone()
        bad[4, e] = value
        got = moe.route_backward(bad, indx, d, "softmax_topk")
        if chosen[e]:
            assert got[4][chosen].isnan().all() and (got[4][~chosen] == 0).all()
            got[4] = clean[4]
        assert torch.equal(got, clean)


@pytest.mark.parametrize("gating", ["softmax_topk", "softmax_all"])
@pytest.mark.parametrize("value", [NAN, INF])
def test_a_gradient_that_is_not_finite(gating, value):
    """Over the selected, the other experts' gradients stay zero."""
    z, indx, d = setup(32)
    clean = moe.route_backward(z, indx, d, gating)
    d[2, 1] = value
    got = moe.route_backward(z, indx, d, gating)
    chosen = torch.zeros(32, dtype=torch.bool, device="cuda")
    chosen[indx[2].long()] = True
    assert not got[2][chosen].isfinite().any()
    if gating == "softmax_topk":
        assert (got[2][~chosen] == 0).all()
    else:
        assert not got[2].isfinite().any()
    got[2] = clean[2]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("gating", ["softmax_topk", "softmax_all"])
def test_masked_logits(gating):
    """-inf is a probability of zero as long as one logit is left; a token with
    none left has no softmax, and its gate weights are NaN too."""
    z, indx, d = setup(16)
    z[1, indx[1, :3].long()] = -INF
    z[5] = -INF
    got = moe.route_backward(z, indx, d, gating)
    zz, up = z.double(), torch.zeros(9, 16, dtype=torch.float64, device="cuda")
    up.scatter_(1, indx.long(), d.double())
    chosen = torch.zeros(9, 16, dtype=torch.bool, device="cuda").scatter_(1, indx.long(), True)
    if gating == "softmax_topk":
        zz = zz.masked_fill(~chosen, -INF)
    p = torch.softmax(zz, 1)
    ref = p * (up - (p * up).sum(1, keepdim=True))
    rows = [0, 1, 2, 3, 4, 6, 7, 8]
    # p: expf 2 ulp, a sum of 16, a division, arguments below 16; then two products
    tol = p * (up.abs() + (p * up.abs()).sum(1, keepdim=True)) * (2 * (2 * 20 + 20) + 8) * 2.0 ** -24
    assert ((got.double() - ref).abs() <= tol + 2.0 ** -140)[rows].all()
    live = chosen[5] if gating == "softmax_topk" else torch.ones_like(chosen[5])
    assert got[5][live].isnan().all() and (got[5][~live] == 0).all()
    _, vals = moe.route(z, 4, gating)
    assert vals[5].isnan().all()
