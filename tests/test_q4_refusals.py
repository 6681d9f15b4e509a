"""What moe_linear_q4, moe_grouped_ffn_q4 and moe_forward_q4 refuse, on the
host and before any launch."""
import ctypes

import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from mixture_experts_routing_warp_gb300 import build as cuda_build
from mixture_experts_routing_warp_gb300._binding import Q4Matrix

BASE = 1 << 20
INVALID, UNSUPPORTED, SMALL, MISALIGNED = 1, 2, 3, 6
REF = object()


@pytest.fixture(scope="module")
def L():
    cuda_build.build()
    return moe.lib()


def q4(codes=BASE, scales=BASE, whole=0, fmt=0):
    return ctypes.byref(Q4Matrix(codes, scales, whole, fmt))


def meta(**spoil):
    m = dict(col_sum=BASE, offs=BASE, col_sorted=BASE, row_sorted=BASE, gate_scal=BASE)
    m.update(spoil)
    return ctypes.byref(moe.RoutingMeta(*m.values()))


def _p(v):
    return ctypes.c_void_p(v)


def linear(L, x=BASE, w=REF, n=4, R=8, C=64, dtype=0, y=BASE):
    return L.moe_linear_q4(_p(x), q4() if w is REF else w, n, R, C, dtype, _p(y), None)


def ffn(L, x=BASE, m=REF, w13=REF, w2=REF, n=4, E=8, k=2, H=64, I=128, p=REF, dtype=0, y=BASE,
        ws=BASE, size=None):
    size = moe.workspace_q4_size(4, 8, 2, 64, 128) if size is None else size
    p = ctypes.byref(moe.make_params()) if p is REF else p
    return L.moe_grouped_ffn_q4(_p(x), meta() if m is REF else m, q4() if w13 is REF else w13,
                                q4() if w2 is REF else w2, n, E, k, H, I, p, dtype, _p(y), _p(ws),
                                size, None)


def forward(L, x=BASE, z=BASE, w13=REF, w2=REF, n=4, E=8, k=2, H=64, I=128, p=REF, dtype=0,
            out=BASE, indx=0, vals=0, m=None, ws=BASE, size=None):
    size = moe.workspace_q4_size(4, 8, 2, 64, 128) if size is None else size
    p = ctypes.byref(moe.make_params()) if p is REF else p
    return L.moe_forward_q4(_p(x), _p(z), q4() if w13 is REF else w13, q4() if w2 is REF else w2,
                            n, E, k, H, I, p, dtype, _p(out), _p(indx), _p(vals), m, _p(ws), size,
                            None)


@pytest.mark.parametrize("spoil", [
    dict(n=-1), dict(n=2 ** 31), dict(R=0), dict(R=2 ** 30 + 1), dict(C=0), dict(C=16), dict(C=48),
    dict(C=2 ** 24 + 32), dict(dtype=2), dict(dtype=-1), dict(x=0), dict(y=0), dict(w=None)])
def test_linear_invalid(L, spoil):
    assert linear(L, **spoil) == INVALID


@pytest.mark.parametrize("call", [linear, ffn, forward])
def test_matrix_arguments(L, call):
    name = "w" if call is linear else "w2"
    for bad in (q4(codes=0), q4(scales=0), q4(fmt=2), q4(fmt=-1)):
        assert call(L, **{name: bad}) == INVALID
    for bad in (q4(codes=BASE + 8), q4(scales=BASE + 2), q4(whole=BASE + 2)):
        assert call(L, **{name: bad}) == MISALIGNED


@pytest.mark.parametrize("call", [ffn, forward])
def test_layer_arguments(L, call):
    for spoil in (dict(n=-1), dict(E=0), dict(E=257), dict(k=0), dict(k=9), dict(H=32),
                  dict(H=96), dict(I=100), dict(n=1 << 30), dict(dtype=2), dict(p=None),
                  dict(w13=None), dict(w2=None), dict(x=0), dict(ws=0)):
        assert call(L, **spoil) == INVALID, spoil
    size = moe.workspace_q4_size(4, 8, 2, 64, 128)
    assert call(L, size=size - 1) == SMALL
    assert call(L, x=BASE + 8) == MISALIGNED
    assert call(L, ws=BASE + 128) == MISALIGNED
    relu = moe.make_params(act="relu2", limit=1.0)
    assert call(L, p=ctypes.byref(relu)) == UNSUPPORTED


def test_ffn_metadata(L):
    assert ffn(L, m=None) == INVALID
    assert ffn(L, m=meta(offs=0)) == INVALID
    assert ffn(L, m=meta(col_sorted=0)) == INVALID
    assert ffn(L, m=meta(offs=BASE + 2)) == MISALIGNED
    assert ffn(L, y=0) == INVALID
    assert ffn(L, y=BASE + 2) == MISALIGNED


def test_forward_outputs_and_map(L):
    assert forward(L, E=1) == INVALID                # k of E experts
    assert forward(L, indx=BASE) == INVALID          # topk outputs come as a pair
    assert forward(L, z=0) == INVALID
    assert forward(L, out=0) == INVALID
    assert forward(L, z=BASE + 2) == MISALIGNED
    assert forward(L, m=meta(row_sorted=0)) == INVALID
    p = moe.make_params()
    p.expert_map = BASE
    for local, rc in ((0, INVALID), (9, INVALID), (8, 0), (1, 0)):
        p.n_local_experts = local
        assert forward(L, p=ctypes.byref(p), n=0) == rc
    p.expert_map = BASE + 2
    assert forward(L, p=ctypes.byref(p), n=0) == MISALIGNED


def test_no_tokens_is_a_no_op(L):
    assert linear(L, n=0, x=0, y=0) == 0
    assert ffn(L, n=0, x=0, y=0, m=meta(col_sorted=0), ws=0, size=0) == 0
    assert forward(L, n=0, x=0, z=0, out=0, ws=0, size=0) == 0


def test_workspace_size():
    assert moe.workspace_q4_size(0, 4, 2, 64, 64) > 0
    for bad in ((-1, 8, 2, 64, 128), (4, 8, 9, 64, 128), (4, 8, 2, 65, 128), (4, 300, 2, 64, 64)):
        assert moe.workspace_q4_size(*bad) == 0
    n, E, k, H, I = 1000, 8, 2, 512, 1408
    assert moe.workspace_q4_size(n, E, k, H, I) >= n * k * (4 * I + 2 * H)


def test_binding_checks():
    codes, scales = torch.zeros(8, 32, dtype=torch.uint8), torch.zeros(8, 2, dtype=torch.uint8)
    with pytest.raises(ValueError, match="fmt"):
        moe.Q4Weight(codes, scales, "int4")
    with pytest.raises(ValueError, match="CUDA"):
        moe.Q4Weight(codes, scales, "mxfp4")
    with pytest.raises(ValueError, match="CUDA"):
        moe.linear_q4(torch.zeros(1, 64, dtype=torch.bfloat16), None)
