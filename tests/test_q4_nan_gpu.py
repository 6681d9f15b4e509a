"""NaN in the experts' 4-bit products (moe.grouped_ffn_q4): the activations
between the products pass it on, clamps and max(a, 0) included."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from test_q4_experts_gpu import ACTS, experts64, weights
from test_q4_gpu import BF16, check, make_meta, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("act,layout,limit", ACTS)
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_nan_reaches_what_it_belongs_to(fmt, act, layout, limit):
    """A NaN activation reaches its token's rows, one in w13 its expert's rows,
    one in w2 its column of the expert's rows, and none of them another."""
    n, H, I, E, k = 7, 128, 192, 3, 2
    w13, w2 = weights(fmt, E, H, I, act, 110)
    meta, clean = make_meta(n, E, k, 112), tokens(n, H, BF16, 113)
    p = moe.make_params(act=act, layout=layout, limit=limit)
    ws, nan = moe.workspace_q4(n, E, k, H, I), 255 if fmt == "mxfp4" else 127
    ref, tol = experts64(clean, meta, w13, w2, k, act, layout, limit)
    offs = meta["offs"].tolist()
    token = meta["col_sorted"].long() // k
    e = max(range(E), key=lambda i: offs[i + 1] - offs[i])
    mine = torch.zeros(n * k, dtype=torch.bool, device="cuda")
    mine[offs[e]:offs[e + 1]] = True
    assert mine.any() and not mine.all()

    def run(x, bad):
        got = moe.grouped_ffn_q4(x, meta, w13, w2, k, ws, p)
        assert got[bad].isnan().all()
        check(got[~bad], ref[~bad], tol[~bad])

    column = torch.zeros(H, dtype=torch.bool, device="cuda")
    whole = torch.ones(H, dtype=torch.bool, device="cuda")
    x = clean.clone()
    x[3, 77] = float("nan")
    run(x, (token == 3)[:, None] & whole)
    for scales, bad in ((w13.scales, mine[:, None] & whole), (w2.scales, None)):
        row = 37
        if bad is None:
            column[row] = True
            bad = mine[:, None] & column
        kept = scales[e, row, 1].clone()
        scales[e, row, 1] = nan
        run(clean, bad)
        scales[e, row, 1] = kept
    if fmt == "nvfp4":
        w13.matrix_scale[e] = float("nan")
        run(clean, mine[:, None] & whole)
