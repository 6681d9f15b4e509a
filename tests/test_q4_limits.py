"""The largest matrix of 4-bit weights, 2^36 codes: what is past it is refused
by every call and has no workspace (host only, no launch)."""
import ctypes

import pytest

import mixture_experts_routing_warp_gb300 as moe
from mixture_experts_routing_warp_gb300 import build as cuda_build
from test_q4_refusals import BASE, INVALID, ffn, forward, linear

H, I = 65536, 1 << 19   # w13 of a gated activation: 2 I H = 2^36 codes


@pytest.fixture(scope="module")
def L():
    cuda_build.build()
    return moe.lib()


def test_layer_calls(L):
    assert moe.workspace_q4_size(1, 8, 2, H, I) > 0
    assert moe.workspace_q4_size(1, 8, 2, H, I + 64) == 0
    for call in (ffn, forward):
        assert call(L, n=0, H=H, I=I) == 0
        assert call(L, n=0, H=H, I=I + 64) == INVALID
        assert call(L, n=1, H=H, I=I + 64, size=1 << 62) == INVALID
        relu = ctypes.byref(moe.make_params(act="relu2"))
        assert call(L, n=0, H=H, I=I + 64, p=relu) == INVALID


def test_linear(L):
    assert linear(L, n=0, R=1 << 22, C=1 << 14) == 0
    assert linear(L, n=0, R=(1 << 22) + 1, C=1 << 14) == INVALID
    assert linear(L, n=0, x=BASE, R=1 << 30, C=96) == INVALID
