"""The experts with 4-bit weights (moe.grouped_ffn_q4): the bits of the
intermediate. Formulas, inputs and roundings as in test_q4_gpu.

h enters the second product as two fp16 terms: the first is off by at most
2^-11 of the value, the second holds the rest to 2^-11 of that, 2^-22 in all;
below fp16's range both stop at half its smallest step, 2^-39 of the row's
largest magnitude."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from test_q4_gpu import (BF16, FP16, activate64, check, decode64, make_meta, product64, random_q4,
                         tokens)

pytestmark = pytest.mark.gpu

ACTS = [("swiglu", "packed", None), ("swiglu", "interleaved", 2.0),
        ("swiglu_oai", "interleaved", None), ("relu2", "packed", None)]


def experts64(x, meta, w13, w2, k, act, layout, limit=None):
    """The sorted outputs and the bound on their error before the last rounding."""
    offs, N = meta["offs"].tolist(), meta["col_sorted"].numel()
    y = torch.zeros(N, x.shape[1], dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    for e in range(len(offs) - 1):
        lo, hi = offs[e], offs[e + 1]
        if lo == hi:
            continue
        tok = meta["col_sorted"][lo:hi].long() // k
        h, eh = activate64(*product64(x[tok].double(), decode64(w13, e)), act, layout, limit)
        W2 = decode64(w2, e)
        y[lo:hi], err = product64(h, W2)
        tol[lo:hi] = err + (eh + 2.0 ** -22 * h.abs()) @ W2.abs().t()
    return y, tol


def weights(fmt, E, H, I, act, seed):
    return (random_q4((I if act == "relu2" else 2 * I, H), fmt, seed, count=E),
            random_q4((H, I), fmt, seed + 1, count=E))


@pytest.mark.parametrize("act,layout,limit", ACTS)
@pytest.mark.parametrize("fmt,scale", [("mxfp4", 30.0), ("nvfp4", 0.3)])
@pytest.mark.parametrize("n", [1, 5, 24])
def test_h_keeps_more_bits_than_the_result(n, fmt, scale, act, layout, limit):
    """fp16 results are those of a nearly exact h, rounded once."""
    H, I, E, k = 256, 512, 4, 2
    w13, w2 = weights(fmt, E, H, I, act, 100)
    meta, x = make_meta(n, E, k, 102), tokens(n, H, FP16, 103, scale)
    ws = moe.workspace_q4(n, E, k, H, I)
    got = moe.grouped_ffn_q4(x, meta, w13, w2, k, ws,
                             moe.make_params(act=act, layout=layout, limit=limit))
    ref, tol = experts64(x, meta, w13, w2, k, act, layout, limit)
    assert ref.abs().max() > 0.01
    check(got, ref, tol)


def test_infinite_activations_of_the_second_product():
    """ReLU2 sends a large product to infinity: its rows of y are infinite or
    NaN as the weights say, other rows are as before."""
    n, H, I, E, k = 6, 64, 64, 2, 1
    w13, w2 = weights("nvfp4", E, H, I, "relu2", 120)
    w2.codes[:, :] = 0x13          # 1.5 and 0.5: no zero weight
    w2.scales.copy_(w2.scales & 127)
    w2.scales.clamp_(8, 100)       # positive
    meta, x = make_meta(n, E, k, 122), tokens(n, H, BF16, 123)
    p, ws = moe.make_params(act="relu2"), moe.workspace_q4(n, E, k, H, I)
    ref, tol = experts64(x, meta, w13, w2, k, "relu2", "packed")
    x[2] *= 2.0 ** 100             # squares past fp32's range
    got = moe.grouped_ffn_q4(x, meta, w13, w2, k, ws, p)
    mine = meta["col_sorted"].long() // k == 2
    assert (got[mine] == float("inf")).all()
    check(got[~mine], ref[~mine], tol[~mine])
