"""What the calls of the dense blocks refuse, on the host and before any launch."""
import ctypes

import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from mixture_experts_routing_warp_gb300 import build as cuda_build

BASE = 1 << 20
INVALID, UNSUPPORTED, SMALL, MISALIGNED = 1, 2, 3, 6
PLENTY = 1 << 40


@pytest.fixture(scope="module")
def L():
    cuda_build.build()
    return moe.lib()


class Ptr(int):
    """An address (never read: each test spoils the call that has it)."""


P = Ptr(BASE)


def rows8(codes=BASE, scales=BASE):
    return ctypes.byref(moe._binding.Mx8Rows(codes, scales))


def params(act="swiglu", **kw):
    return ctypes.byref(moe.make_params(act=act, **kw))


CALLS = {
    "moe_rms_norm": dict(x=P, residual=P, weight=P, wdtype=2, n=4, H=64, dtype=0, eps=1e-5, y=P,
                         y8=None, sum=P),
    "moe_rms_norm_backward": dict(d_y=P, x=P, weight=P, wdtype=2, d_sum=P, n=4, H=64, dtype=0,
                                  eps=1e-5, d_x=P, d_weight=P, ws=P, bytes=PLENTY),
    "moe_linear": dict(x=P, w=P, bias=P, residual=P, n=100, R=64, C=2880, dtype=0, act=1, y=P,
                       ws=P, bytes=PLENTY, status=P),
    "moe_linear_mx8": dict(x8=rows8(), w8=rows8(), bias=P, residual=P, n=40, R=64, C=64, dtype=0,
                           act=0, y=P, ws=P, bytes=PLENTY, status=P),
    "moe_linear_backward": dict(d_y=P, x=P, w=P, bias=P, n=4, R=64, C=64, dtype=0, act=1, d_x=P,
                                d_w=P, d_bias=P, ws=P, bytes=PLENTY, status=P),
    "moe_gated_linear": dict(x=P, w13=P, n=100, H=2880, I=64, params=params(), dtype=0, h=P,
                             h8=None, ws=P, bytes=PLENTY, status=P),
    "moe_gated_linear_mx8": dict(x8=rows8(), w8=rows8(), n=40, H=64, I=64, params=params(),
                                 dtype=0, h=None, h8=rows8(), ws=P, bytes=PLENTY, status=P),
    "moe_gated_linear_backward": dict(d_h=P, x=P, w13=P, n=4, H=64, I=64, params=params(),
                                      dtype=0, d_x=P, d_w13=P, ws=P, bytes=PLENTY, status=P),
}
OPTIONAL = {"residual", "weight", "sum", "d_sum", "d_weight", "bias", "status", "d_x", "d_w",
            "d_bias", "d_w13"}


def call(L, name, **spoil):
    args = dict(CALLS[name], **spoil)
    return getattr(L, name)(*[ctypes.c_void_p(int(v)) if isinstance(v, Ptr) else v
                              for v in args.values()], None)


SPOILED = [(name, s) for name in CALLS for s in (
    [{"n": -1}, {"n": 1 << 31}, {"dtype": -1}, {"dtype": 3}] +
    [{"eps": e} for e in (-1.0, float("nan"), float("inf")) if "eps" in CALLS[name]] +
    [{"wdtype": d} for d in (1, 3, -1) if "wdtype" in CALLS[name]] +
    [{"act": a} for a in (-1, 4) if "act" in CALLS[name]] +
    [{"C": c} for c in (0, -8, 65544, 4) if "C" in CALLS[name]] +
    [{"R": r} for r in (0, -8, 131080) if "R" in CALLS[name]] +
    [{"I": i} for i in (0, 4, 12, 65544) if "I" in CALLS[name]] +
    [{"H": h} for h in (0, -64, 65600) if "H" in CALLS[name]])]
SPOILED += [("moe_linear_backward", {"R": 12}), ("moe_linear", {"dtype": 2}),
            ("moe_linear", {"n": 1 << 30, "C": 1024}),          # 2^40 elements
            ("moe_linear_mx8", {"C": 40}), ("moe_gated_linear_mx8", {"H": 40}),
            ("moe_gated_linear", {"H": 12}), ("moe_gated_linear_backward", {"H": 4}),
            ("moe_gated_linear_mx8", {"I": 40}),                 # groups of 32 in the result
            ("moe_rms_norm", {"H": 40, "y": None, "y8": rows8()}),
            ("moe_rms_norm", {"residual": None})]                # a sum without a residual


@pytest.mark.parametrize("name,spoil", SPOILED)
def test_sizes_and_enums(L, name, spoil):
    assert call(L, name, **spoil) == INVALID


def test_one_result(L):
    """Exactly one of the 16-bit and the 8-bit result."""
    assert call(L, "moe_rms_norm", y=None) == INVALID
    assert call(L, "moe_rms_norm", y8=rows8()) == INVALID
    for name in ("moe_gated_linear", "moe_gated_linear_mx8"):
        assert call(L, name, h=None, h8=None) == INVALID
        assert call(L, name, h=P, h8=rows8()) == INVALID


@pytest.mark.parametrize("name", CALLS)
def test_null_and_misaligned_pointers(L, name):
    for arg, v in CALLS[name].items():
        if not isinstance(v, Ptr):
            continue
        if arg == "ws":
            assert call(L, name, ws=None) == INVALID
            assert call(L, name, ws=Ptr(BASE + 16)) == MISALIGNED
            assert call(L, name, bytes=1) == SMALL
            continue
        if arg not in OPTIONAL:
            assert call(L, name, **{arg: None}) == INVALID, arg
        assert call(L, name, **{arg: Ptr(BASE + 1)}) == MISALIGNED, arg
        if arg in ("x", "w", "w13", "d_x", "d_w", "d_w13") and "norm" not in name or \
                (name, arg) == ("moe_linear_backward", "d_y"):
            assert call(L, name, **{arg: Ptr(BASE + 8)}) == MISALIGNED, arg
    for arg in ("x8", "w8"):
        if arg in CALLS[name]:
            assert call(L, name, **{arg: None}) == INVALID
            assert call(L, name, **{arg: rows8(codes=None)}) == INVALID
            assert call(L, name, **{arg: rows8(scales=None)}) == INVALID
            assert call(L, name, **{arg: rows8(codes=BASE + 8)}) == MISALIGNED


@pytest.mark.parametrize("name", [n for n in CALLS if "gated" in n])
def test_activation(L, name):
    assert call(L, name, params=None) == INVALID
    assert call(L, name, params=params("relu2")) == UNSUPPORTED   # it has no gate
    assert call(L, name, params=params(limit=-1.0)) == INVALID


@pytest.mark.parametrize("name", CALLS)
def test_no_rows_is_a_no_op(L, name):
    empty = {a: None for a, v in CALLS[name].items() if isinstance(v, Ptr) or a in ("x8", "w8")}
    assert call(L, name, n=0, **empty) == 0


def test_workspace_sizes(L):
    assert moe.linear_workspace_size(8, 2880, 2880) == 0          # few rows
    assert moe.linear_workspace_size(8192, 2880, 2880) == 0       # more tiles than SMs
    assert moe.linear_workspace_size(200, 256, 8192) > 0          # a split sum
    assert moe.linear_workspace_size(8, 64, 64, True) == 0
    assert moe.linear_workspace_size(40, 64, 64, True) > 0        # scales laid out
    assert moe.gated_linear_workspace_size(8, 64, 64) == 0
    assert moe.gated_linear_workspace_size(8, 64, 64, True, True) == 0
    assert moe.gated_linear_workspace_size(40, 64, 64, True, True) > 0
    assert moe.rms_norm_backward_workspace_size(8, 64) > 0
    assert moe.linear_backward_workspace_size(64, 64, 64) >= 0
    for bad in ((8, 64, 60), (-1, 64, 64), (8, 0, 64)):
        assert moe.linear_workspace_size(*bad) == 0
    assert moe.linear_backward_workspace_size(8, 60, 64) == 0
    assert moe.gated_linear_backward_workspace_size(8, 64, 60) == 0
    with pytest.raises(KeyError):
        moe.linear_backward_workspace_size(8, 64, 64, "tanh")


def test_binding_checks():
    x, w = torch.zeros(4, 64, dtype=torch.bfloat16), torch.zeros(8, 64, dtype=torch.bfloat16)
    p = moe.make_params()
    for fn in (lambda: moe.rms_norm(x, None), lambda: moe.rms_norm_backward(x, x, None),
               lambda: moe.linear(x, w), lambda: moe.linear_backward(x, x, w),
               lambda: moe.gated_linear(x, w, p), lambda: moe.gated_linear_backward(x, x, w, p),
               lambda: moe.Mx8(x.to(torch.float8_e4m3fn), torch.zeros(4, 2, dtype=torch.uint8))):
        with pytest.raises(ValueError, match="CUDA|cuda"):
            fn()
    with pytest.raises(ValueError, match="bfloat16, float16 or float32"):
        moe.linear(x.double(), w)
    with pytest.raises(ValueError, match="act must be one of"):
        moe.linear(x, w, act="tanh")
    with pytest.raises(ValueError):
        moe.linear([1.0], w)
    with pytest.raises(ValueError):
        moe.Mx8([1.0], [1.0])
