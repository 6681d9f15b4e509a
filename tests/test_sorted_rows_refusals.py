"""What moe_dispatch, moe_combine_weighted, their gradients and
moe_route_backward refuse, on the host and before any launch."""
import ctypes

import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from mixture_experts_routing_warp_gb300 import build as cuda_build

BASE = 1 << 20
INVALID, MISALIGNED = 1, 6


@pytest.fixture(scope="module")
def L():
    cuda_build.build()
    return moe.lib()


def _p(v):
    return ctypes.c_void_p(v)


# name -> arguments of a call that would launch (never made: each test spoils one)
CALLS = {
    "moe_dispatch": dict(x=BASE, row_sorted=BASE, n_kept=BASE, n=4, k=2, H=64, dtype=0,
                         x_sorted=BASE),
    "moe_dispatch_backward": dict(d_sorted=BASE, row_sorted=BASE, n=4, k=2, H=64, dtype=0,
                                  d_x=BASE),
    "moe_combine_weighted": dict(y_sorted=BASE, row_sorted=BASE, weights=BASE, wdtype=2, n=4, k=2,
                                 H=64, dtype=0, out=BASE),
    "moe_combine_weighted_backward": dict(d_out=BASE, y_sorted=BASE, row_sorted=BASE,
                                          weights=BASE, wdtype=2, n_kept=BASE, n=4, k=2, H=64,
                                          dtype=0, d_sorted=BASE, d_weights=BASE),
    "moe_route_backward": dict(logits=BASE, topk_indx=BASE, d_vals=BASE, n=4, E=8, k=2, gating=0,
                               d_logits=BASE),
}
SIZES = ("n", "k", "H", "E", "dtype", "wdtype", "gating")


def call(L, name, **spoil):
    args = dict(CALLS[name], **spoil)
    return getattr(L, name)(*[v if a in SIZES else _p(v) for a, v in args.items()], None)


SPOILED = [(name, {"n": -1}) for name in CALLS] + [(name, {"k": k}) for name in CALLS
                                                    for k in (0, 9)] + \
          [(name, {"n": 1 << 30}) for name in CALLS] + \
          [(name, {"H": H}) for name in CALLS if "H" in CALLS[name] for H in (0, -64, 65537)] + \
          [(name, {"dtype": d}) for name in CALLS if "dtype" in CALLS[name] for d in (-1, 3)] + \
          [(name, {"wdtype": d}) for name in CALLS if "wdtype" in CALLS[name] for d in (1, 3)] + \
          [("moe_route_backward", s) for s in ({"E": 0}, {"E": 257}, {"E": 1}, {"gating": 2})]


@pytest.mark.parametrize("name,spoil", SPOILED)
def test_sizes_and_enums(L, name, spoil):
    assert call(L, name, **spoil) == INVALID


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned_pointers(L, name):
    for arg in CALLS[name]:
        if arg in SIZES:
            continue
        if arg != "n_kept":   # the one optional array
            assert call(L, name, **{arg: 0}) == INVALID, arg
        assert call(L, name, **{arg: BASE + 1}) == MISALIGNED, arg
        if arg in ("row_sorted", "n_kept", "d_weights", "topk_indx", "d_vals", "logits",
                   "d_logits", "weights"):
            assert call(L, name, **{arg: BASE + 2}) == MISALIGNED, arg


@pytest.mark.parametrize("name", CALLS)
def test_no_tokens_is_a_no_op(L, name):
    empty = {a: 0 for a in CALLS[name] if a not in SIZES}
    assert call(L, name, n=0, **empty) == 0


def test_binding_checks():
    meta = {"row_sorted": torch.zeros(8, dtype=torch.int32),
            "offs": torch.zeros(5, dtype=torch.int32)}
    x, y, w = torch.zeros(4, 64), torch.zeros(8, 64), torch.zeros(4, 2)
    for fn in (lambda: moe.dispatch(x, meta, 2), lambda: moe.dispatch_backward(y, meta, 2),
               lambda: moe.combine_weighted(y, meta, w),
               lambda: moe.combine_weighted_backward(x, y, meta, w),
               lambda: moe.route_backward(torch.zeros(4, 8), meta["row_sorted"].view(4, 2), w)):
        with pytest.raises(ValueError, match="CUDA"):
            fn()
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        moe.dispatch(x.double(), meta, 2)
