"""ctypes binding over the C ABI in include/moe.h (argument marshalling only).

Every stage runs in the CUDA library libmoe_gb300.so; this module checks
tensor devices / dtypes / shapes, allocates outputs with PyTorch, passes
`data_ptr()`s and the current CUDA stream, and turns a non-zero moe_status
into an exception. There is no fallback: if the library is missing, every
call raises.
"""
from __future__ import annotations

import ctypes
import functools
import math
import os
from typing import Optional

import torch

from . import build as _build

GATING = {"softmax_topk": 0, "softmax_all": 1}
ACT = {"swiglu": 0, "swiglu_oai": 1, "relu2": 2}
LAYOUT = {"packed": 0, "interleaved": 1}
SET_ALPHA, SET_BETA, SET_LIMIT = 1, 2, 4
FFN_KERNEL = {"auto": 0, "tiled": 1, "swap": 2}
Q4_FORMAT = {"mxfp4": 0, "nvfp4": 1}
Q4_GROUP = {"mxfp4": 32, "nvfp4": 16}
LINEAR_ACT = {"none": 0, "silu": 1, "gelu": 2, "relu2": 3}
DTYPE = {torch.bfloat16: 0, torch.float16: 1, torch.float32: 2}
ABI_VERSION = 4

STATUS = {0: "MOE_OK", 1: "MOE_ERR_INVALID_ARG", 2: "MOE_ERR_UNSUPPORTED",
          3: "MOE_ERR_WORKSPACE_TOO_SMALL", 4: "MOE_ERR_CUDA", 5: "MOE_ERR_TIMEOUT",
          6: "MOE_ERR_MISALIGNED"}


class MoEError(RuntimeError):
    def __init__(self, status: int, what: str):
        super().__init__(f"{what}: {STATUS.get(status, status)}")
        self.status = status


class MoeParams(ctypes.Structure):
    _fields_ = [("gating", ctypes.c_int32), ("activation", ctypes.c_int32),
                ("w13_layout", ctypes.c_int32), ("set", ctypes.c_uint32),
                ("alpha", ctypes.c_float), ("beta", ctypes.c_float), ("limit", ctypes.c_float),
                ("ffn_kernel", ctypes.c_int32), ("expert_map", ctypes.c_void_p),
                ("n_local_experts", ctypes.c_int32)]


class RoutingMeta(ctypes.Structure):
    _fields_ = [("col_sum", ctypes.c_void_p), ("offs", ctypes.c_void_p),
                ("col_sorted", ctypes.c_void_p), ("row_sorted", ctypes.c_void_p),
                ("gate_scal", ctypes.c_void_p)]


class Q4Matrix(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p),
                ("matrix_scale", ctypes.c_void_p), ("format", ctypes.c_int32)]


class Mx8Rows(ctypes.Structure):
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p)]


_LIB = None

# name -> (restype, argtypes)
_P, _I64, _I32, _SZ, _U64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                             ctypes.c_uint64)
_PP = ctypes.POINTER(MoeParams)
_PM = ctypes.POINTER(RoutingMeta)
_PQ = ctypes.POINTER(Q4Matrix)
_P8 = ctypes.POINTER(Mx8Rows)
_F32 = ctypes.c_float
SIGNATURES = {
    "moe_abi_version": (_I32, []),
    "moe_status_string": (ctypes.c_char_p, [_I32]),
    "moe_workspace_size": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_workspace_init": (_I32, [_P, _SZ, _P]),
    "moe_workspace_regions": (_I32, [_I64, _I32, _I32, _I32, _I32, _P, _P]),
    "moe_route": (_I32, [_P, _I64, _I32, _I32, _I32, _P, _P, _P]),
    "moe_build_metadata": (_I32, [_P, _P, _I64, _I32, _I32, _PM, _P, _SZ, _P]),
    "moe_route_metadata": (_I32, [_P, _I64, _I32, _I32, _I32, _P, _P, _PM, _P, _SZ, _P]),
    "moe_build_metadata_noalloc": (_I32, [_P, _P, _I64, _I32, _I32, _PM, _P, _P]),
    "moe_grouped_ffn": (_I32, [_P, _PM, _P, _P, _I64, _I32, _I32, _I32, _I32, _PP, _P, _P, _SZ,
                               _P]),
    "moe_combine": (_I32, [_P, _I64, _I32, _I32, _P, _P]),
    "moe_forward": (_I32, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _PP, _P, _P, _P, _PM,
                           _P, _SZ, _P]),
    "moe_forward_timed": (_I32, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _PP, _P, _P, _P,
                                 _PM, _P, _SZ, _P, _I32, _P]),
    "moe_route_gemm": (_I32, [_P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P, _SZ, _P]),
    "moe_forward_gate": (_I32, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _PP, _P, _P, _P,
                                _PM, _P, _SZ, _P]),
    "moe_forward_launch_count": (_I32, [_I64, _I32, _I32, _I32, _I32]),
    "moe_ffn_plan": (_I32, [_I64, _I32, _I32, _I32, _I32, _P, _P]),
    "moe_dispatch": (_I32, [_P, _P, _P, _I64, _I32, _I32, _I32, _P, _P]),
    "moe_dispatch_backward": (_I32, [_P, _P, _I64, _I32, _I32, _I32, _P, _P]),
    "moe_combine_weighted": (_I32, [_P, _P, _P, _I32, _I64, _I32, _I32, _I32, _P, _P]),
    "moe_combine_weighted_backward": (_I32, [_P, _P, _P, _P, _I32, _P, _I64, _I32, _I32, _I32, _P,
                                             _P, _P]),
    "moe_route_backward": (_I32, [_P, _P, _P, _I64, _I32, _I32, _I32, _P, _P]),
    "moe_linear_q4": (_I32, [_P, _PQ, _I64, _I32, _I32, _I32, _P, _P]),
    "moe_q4_workspace_size": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_grouped_ffn_q4": (_I32, [_P, _PM, _PQ, _PQ, _I64, _I32, _I32, _I32, _I32, _PP, _I32, _P,
                                  _P, _SZ, _P]),
    "moe_forward_q4": (_I32, [_P, _P, _PQ, _PQ, _I64, _I32, _I32, _I32, _I32, _PP, _I32, _P, _P,
                              _P, _PM, _P, _SZ, _P]),
    "moe_rms_norm": (_I32, [_P, _P, _P, _I32, _I64, _I32, _I32, _F32, _P, _P8, _P, _P]),
    "moe_rms_norm_backward_workspace_size": (_SZ, [_I64, _I32]),
    "moe_rms_norm_backward": (_I32, [_P, _P, _P, _I32, _P, _I64, _I32, _I32, _F32, _P, _P, _P,
                                     _SZ, _P]),
    "moe_linear_workspace_size": (_SZ, [_I64, _I32, _I32, _I32]),
    "moe_linear": (_I32, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _SZ, _P, _P]),
    "moe_linear_mx8": (_I32, [_P8, _P8, _P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _SZ, _P,
                              _P]),
    "moe_linear_backward_workspace_size": (_SZ, [_I64, _I32, _I32, _I32]),
    "moe_linear_backward": (_I32, [_P, _P, _P, _P, _I64, _I32, _I32, _I32, _I32, _P, _P, _P, _P,
                                   _SZ, _P, _P]),
    "moe_gated_linear_workspace_size": (_SZ, [_I64, _I32, _I32, _I32, _I32]),
    "moe_gated_linear": (_I32, [_P, _P, _I64, _I32, _I32, _PP, _I32, _P, _P8, _P, _SZ, _P, _P]),
    "moe_gated_linear_mx8": (_I32, [_P8, _P8, _I64, _I32, _I32, _PP, _I32, _P, _P8, _P, _SZ, _P,
                                    _P]),
    "moe_gated_linear_backward_workspace_size": (_SZ, [_I64, _I32, _I32]),
    "moe_gated_linear_backward": (_I32, [_P, _P, _P, _I64, _I32, _I32, _PP, _I32, _P, _P, _P,
                                         _SZ, _P, _P]),
    "moe_read_status": (_I32, [_P, _SZ, _I32, _P]),
    "moe_read_dense_status": (_I32, [_I32, _P]),
    "moe_selftest_wait_timeout": (_I32, [_P, _SZ, _U64, _P]),
    "moe_selftest_linear_timeout": (_I32, [_P, _P, _I64, _I32, _I32, _I32, _P, _P, _SZ, _U64, _P,
                                           _P]),
}


def library_path() -> str:
    return _build.LIB


def lib() -> ctypes.CDLL:
    """Load libmoe_gb300.so (built by `__graft_entry__.build()` or
    `python -m mixture_experts_routing_warp_gb300.build`). Raises if absent."""
    global _LIB
    if _LIB is None:
        path = library_path()
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build the CUDA library first "
                               "(python -m mixture_experts_routing_warp_gb300.build)")
        L = ctypes.CDLL(path)
        for name, (res, args) in SIGNATURES.items():
            f = getattr(L, name)
            f.restype = res
            f.argtypes = args
        if L.moe_abi_version() != ABI_VERSION:
            raise RuntimeError("libmoe_gb300.so ABI version mismatch")
        _LIB = L
    return _LIB


def _check(status: int, what: str) -> None:
    if status != 0:
        raise MoEError(status, what)


def _stream(device: torch.device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t: torch.Tensor, name: str, dtype: torch.dtype, shape=None) -> None:
    if not isinstance(t, torch.Tensor) or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype}, got {t.dtype}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")


def _ptr(t: Optional[torch.Tensor]) -> ctypes.c_void_p:
    return ctypes.c_void_p(0 if t is None else t.data_ptr())


def make_params(gating: str = "softmax_topk", act: str = "swiglu", layout: str = "packed",
                alpha: Optional[float] = None, beta: Optional[float] = None,
                limit: Optional[float] = None, ffn_kernel: str = "auto",
                expert_map: Optional[torch.Tensor] = None,
                n_local_experts: Optional[int] = None) -> MoeParams:
    """moe_params with the `set` bits of the values that are not None, so
    unset parameters keep the activation's defaults. ffn_kernel picks the
    grouped-GEMM kernel: "auto", "tiled" (large per-expert batches) or
    "swap" (small ones). expert_map (int32 [E] on the device: local expert id
    or -1) and n_local_experts make moe_forward compute an expert-parallel
    rank's share; the params keep a reference to the map tensor."""
    p = MoeParams(GATING[gating], ACT[act], LAYOUT[layout], 0, 0.0, 0.0, 0.0,
                  FFN_KERNEL[ffn_kernel], None, 0)
    if expert_map is not None:
        _need(expert_map, "expert_map", torch.int32)
        if n_local_experts is None:
            raise ValueError("an expert map needs n_local_experts")
        p.expert_map = expert_map.data_ptr()
        p.n_local_experts = int(n_local_experts)
        p._map_tensor = expert_map
    if alpha is not None:
        p.set |= SET_ALPHA
        p.alpha = float(alpha)
    if beta is not None:
        p.set |= SET_BETA
        p.beta = float(beta)
    if limit is not None:
        p.set |= SET_LIMIT
        p.limit = float(limit)
    return p


def status_string(status: int) -> str:
    return lib().moe_status_string(int(status)).decode()


def workspace_size(n: int, E: int, k: int, H: int, I: int) -> int:
    return int(lib().moe_workspace_size(n, E, k, H, I))


WS_REGIONS = ("ctrl", "frows", "hist", "topk_indx", "topk_vals", "col_sum", "offs", "col_sorted",
              "row_sorted", "gate_scal", "sync", "sk_part", "x_sorted", "h", "y_flat")


def workspace_regions(n: int, E: int, k: int, H: int, I: int) -> dict:
    """name -> (byte offset, bytes used) of each workspace region."""
    off = (ctypes.c_size_t * len(WS_REGIONS))()
    used = (ctypes.c_size_t * len(WS_REGIONS))()
    _check(lib().moe_workspace_regions(n, E, k, H, I, off, used), "moe_workspace_regions")
    return {name: (int(off[i]), int(used[i])) for i, name in enumerate(WS_REGIONS)}


def workspace(n: int, E: int, k: int, H: int, I: int,
              device: Optional[torch.device] = None) -> torch.Tensor:
    """Allocate (with PyTorch) and initialise a workspace for these sizes."""
    size = workspace_size(n, E, k, H, I)
    if size == 0:
        raise ValueError("invalid sizes for moe_workspace_size")
    device = torch.device("cuda") if device is None else torch.device(device)
    ws = torch.empty(size, dtype=torch.uint8, device=device)
    _check(lib().moe_workspace_init(_ptr(ws), size, _stream(ws.device)), "moe_workspace_init")
    return ws


def route(logits: torch.Tensor, k: int, gating: str = "softmax_topk"):
    """Router top-k -> (topk_indx int32 [n, k], topk_vals bf16 [n, k])."""
    _need(logits, "logits", torch.float32)
    n, E = logits.shape
    indx = torch.empty((n, k), dtype=torch.int32, device=logits.device)
    vals = torch.empty((n, k), dtype=torch.bfloat16, device=logits.device)
    _check(lib().moe_route(_ptr(logits), n, E, k, GATING[gating], _ptr(indx), _ptr(vals),
                           _stream(logits.device)), "moe_route")
    return indx, vals


def empty_meta(N: int, E: int, device) -> dict:
    return {"col_sum": torch.empty(E, dtype=torch.int32, device=device),
            "offs": torch.empty(E + 1, dtype=torch.int32, device=device),
            "col_sorted": torch.empty(N, dtype=torch.int32, device=device),
            "row_sorted": torch.empty(N, dtype=torch.int32, device=device),
            "gate_scal": torch.empty(N, dtype=torch.bfloat16, device=device)}


def _meta_struct(m: dict) -> RoutingMeta:
    return RoutingMeta(m["col_sum"].data_ptr(), m["offs"].data_ptr(), m["col_sorted"].data_ptr(),
                       m["row_sorted"].data_ptr(), m["gate_scal"].data_ptr())


def build_metadata(topk_indx: torch.Tensor, topk_vals: torch.Tensor, E: int,
                   ws: torch.Tensor, meta: Optional[dict] = None) -> dict:
    """Routing metadata -> dict(col_sum, offs, col_sorted, row_sorted,
    gate_scal). gather = (col_sorted, row_sorted), scatter = (row_sorted, col_sorted)."""
    _need(topk_indx, "topk_indx", torch.int32)
    n, k = topk_indx.shape
    _need(topk_vals, "topk_vals", torch.bfloat16, (n, k))
    m = meta if meta is not None else empty_meta(n * k, E, topk_indx.device)
    _check(lib().moe_build_metadata(_ptr(topk_indx), _ptr(topk_vals), n, E, k,
                                    ctypes.byref(_meta_struct(m)), _ptr(ws), ws.numel(),
                                    _stream(topk_indx.device)), "moe_build_metadata")
    return m


def route_metadata(logits: torch.Tensor, k: int, E: Optional[int] = None,
                   gating: str = "softmax_topk", ws: Optional[torch.Tensor] = None,
                   meta: Optional[dict] = None, topk: Optional[tuple] = None):
    """Stages 1 + 2 in one call -> (topk_indx, topk_vals, meta dict)."""
    _need(logits, "logits", torch.float32)
    n, E = logits.shape
    if ws is None:
        ws = workspace(max(n, 1), E, k, 64, 64, logits.device)
    indx, vals = topk if topk is not None else (
        torch.empty((n, k), dtype=torch.int32, device=logits.device),
        torch.empty((n, k), dtype=torch.bfloat16, device=logits.device))
    m = meta if meta is not None else empty_meta(n * k, E, logits.device)
    _check(lib().moe_route_metadata(_ptr(logits), n, E, k, GATING[gating], _ptr(indx), _ptr(vals),
                                    ctypes.byref(_meta_struct(m)), _ptr(ws), ws.numel(),
                                    _stream(logits.device)), "moe_route_metadata")
    return indx, vals, m


def _intermediate(w13: torch.Tensor, params: MoeParams) -> int:
    """I from w13's rows: 2I for the gated activations, I for ReLU2."""
    rows = w13.shape[1]
    return rows if params.activation == ACT["relu2"] else rows // 2


def grouped_ffn(x: torch.Tensor, meta: dict, w13: torch.Tensor, w2: torch.Tensor, k: int,
                ws: torch.Tensor, params: MoeParams,
                y_flat: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gate-weighted per-expert FFN -> y_flat bf16 [n*k, H] in token-slot order."""
    _need(x, "x", torch.bfloat16)
    n, H = x.shape
    _need(w13, "w13", torch.bfloat16)
    E = w13.shape[0]
    I = _intermediate(w13, params)
    _need(w13, "w13", torch.bfloat16, (E, w13.shape[1], H))
    _need(w2, "w2", torch.bfloat16, (E, H, I))
    if y_flat is None:
        y_flat = torch.empty((n * k, H), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_grouped_ffn(_ptr(x), ctypes.byref(_meta_struct(meta)), _ptr(w13), _ptr(w2),
                                 n, E, k, H, I, ctypes.byref(params), _ptr(y_flat),
                                 _ptr(ws), ws.numel(), _stream(x.device)), "moe_grouped_ffn")
    return y_flat


def combine(y_flat: torch.Tensor, n: int, k: int,
            out: Optional[torch.Tensor] = None) -> torch.Tensor:
    _need(y_flat, "y_flat", torch.bfloat16)
    H = y_flat.shape[1]
    if out is None:
        out = torch.empty((n, H), dtype=torch.bfloat16, device=y_flat.device)
    _check(lib().moe_combine(_ptr(y_flat), n, k, H, _ptr(out), _stream(y_flat.device)),
           "moe_combine")
    return out


def forward(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor, k: int,
            params: MoeParams, ws: torch.Tensor, out: Optional[torch.Tensor] = None,
            topk: Optional[tuple] = None, meta: Optional[dict] = None) -> torch.Tensor:
    """The whole layer in one library call. `topk` = (indx, vals) and `meta`
    (dict of the five arrays) are optional outputs."""
    _need(x, "x", torch.bfloat16)
    n, H = x.shape
    _need(logits, "logits", torch.float32)
    E = logits.shape[1]
    E_w = params.n_local_experts if params.expert_map else E  # experts held in w13 / w2
    _need(w13, "w13", torch.bfloat16)
    I = _intermediate(w13, params)
    _need(w13, "w13", torch.bfloat16, (E_w, w13.shape[1], H))
    _need(w2, "w2", torch.bfloat16, (E_w, H, I))
    if out is None:
        out = torch.empty((n, H), dtype=torch.bfloat16, device=x.device)
    indx, vals = topk if topk is not None else (None, None)
    mstruct = ctypes.byref(_meta_struct(meta)) if meta is not None else None
    _check(lib().moe_forward(_ptr(x), _ptr(logits), _ptr(w13), _ptr(w2), n, E, k, H, I,
                             ctypes.byref(params), _ptr(out), _ptr(indx), _ptr(vals), mstruct,
                             _ptr(ws), ws.numel(), _stream(x.device)), "moe_forward")
    return out


def route_gemm(x: torch.Tensor, w_gate: torch.Tensor, k: int, gating: str = "softmax_topk",
               ws: Optional[torch.Tensor] = None, logits: Optional[torch.Tensor] = None):
    """Router matmul x . w_gate^T fused with the top-k -> (topk_indx, topk_vals);
    fills `logits` (fp32 [n, E]) too when given."""
    _need(x, "x", torch.bfloat16)
    n, H = x.shape
    _need(w_gate, "w_gate", torch.bfloat16)
    E = w_gate.shape[0]
    _need(w_gate, "w_gate", torch.bfloat16, (E, H))
    if logits is not None:
        _need(logits, "logits", torch.float32, (n, E))
    if ws is None:
        ws = workspace(max(n, 1), E, k, 64, 64, x.device)
    indx = torch.empty((n, k), dtype=torch.int32, device=x.device)
    vals = torch.empty((n, k), dtype=torch.bfloat16, device=x.device)
    _check(lib().moe_route_gemm(_ptr(x), _ptr(w_gate), n, E, H, k, GATING[gating], _ptr(indx),
                                _ptr(vals), _ptr(logits), _ptr(ws), ws.numel(),
                                _stream(x.device)), "moe_route_gemm")
    return indx, vals


def forward_gate(x: torch.Tensor, w_gate: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                 k: int, params: MoeParams, ws: torch.Tensor, out: Optional[torch.Tensor] = None,
                 topk: Optional[tuple] = None, meta: Optional[dict] = None) -> torch.Tensor:
    """forward() with the routing computed from x and the gate weights [E, H]."""
    _need(x, "x", torch.bfloat16)
    n, H = x.shape
    _need(w_gate, "w_gate", torch.bfloat16)
    E = w_gate.shape[0]
    _need(w_gate, "w_gate", torch.bfloat16, (E, H))
    E_w = params.n_local_experts if params.expert_map else E  # experts held in w13 / w2
    _need(w13, "w13", torch.bfloat16)
    I = _intermediate(w13, params)
    _need(w13, "w13", torch.bfloat16, (E_w, w13.shape[1], H))
    _need(w2, "w2", torch.bfloat16, (E_w, H, I))
    if out is None:
        out = torch.empty((n, H), dtype=torch.bfloat16, device=x.device)
    indx, vals = topk if topk is not None else (None, None)
    mstruct = ctypes.byref(_meta_struct(meta)) if meta is not None else None
    _check(lib().moe_forward_gate(_ptr(x), _ptr(w_gate), _ptr(w13), _ptr(w2), n, E, k, H, I,
                                  ctypes.byref(params), _ptr(out), _ptr(indx), _ptr(vals),
                                  mstruct, _ptr(ws), ws.numel(), _stream(x.device)),
           "moe_forward_gate")
    return out


def _need_on(t: torch.Tensor, name: str, dtype: torch.dtype, device: int, shape=None) -> None:
    """_need, and on the CUDA device of that index (a few hundred ns when all is well)."""
    if not (isinstance(t, torch.Tensor) and t.dtype is dtype and t.get_device() == device >= 0
            and t.is_contiguous() and (shape is None or t.shape == shape)):
        _need(t, name, dtype, shape)
        raise ValueError(f"{name} is on {t.device}, not on cuda:{device}")


def _need_rows(t: torch.Tensor, name: str) -> int:
    """A row tensor [rows, H] of one of the row types; its device's index."""
    if not isinstance(t, torch.Tensor) or t.dtype not in DTYPE:
        raise ValueError(f"{name} must be a bfloat16, float16 or float32 tensor")
    device = t.get_device()
    if device < 0 or not t.is_contiguous():
        _need_on(t, name, t.dtype, device)
    if t.dim() != 2 or t.shape[1] == 0:
        raise ValueError(f"{name} must have shape [rows, H], got {tuple(t.shape)}")
    return device


def _need_slots(meta: dict, slots: int, device: int) -> None:
    """The metadata entries that the row calls read: row_sorted and offs."""
    _need_on(meta["row_sorted"], "row_sorted", torch.int32, device, (slots,))
    offs = meta["offs"]
    _need_on(offs, "offs", torch.int32, device)
    if offs.dim() != 1 or offs.shape[0] < 2:
        raise ValueError("offs must have one entry per expert and one more")


def _kept(meta: dict) -> int:
    """Device address of the number of kept slots: the last offset."""
    offs = meta["offs"]
    return offs.data_ptr() + 4 * (offs.shape[0] - 1)


def _need_weights(weights: torch.Tensor, device: int) -> None:
    if not isinstance(weights, torch.Tensor) or weights.dtype not in (torch.bfloat16,
                                                                      torch.float32):
        raise ValueError("weights must be a bfloat16 or float32 tensor")
    _need_on(weights, "weights", weights.dtype, device)
    if weights.dim() != 2:
        raise ValueError(f"weights must have shape [n, k], got {tuple(weights.shape)}")


def _out_rows(out: Optional[torch.Tensor], name: str, shape, like: torch.Tensor) -> torch.Tensor:
    if out is None:
        return like.new_empty(shape)
    _need_on(out, name, like.dtype, like.get_device(), shape)
    return out


def _run(name: str, device: int, *args) -> None:
    """The library call `name`(*args, stream) on the device's current stream,
    with that device current."""
    fn = getattr(_LIB or lib(), name)
    if device == torch._C._cuda_getDevice():
        status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    else:
        with torch.cuda.device(device):
            status = fn(*args, torch._C._cuda_getCurrentRawStream(device))
    if status != 0:
        raise MoEError(status, name)


def dispatch(x: torch.Tensor, meta: dict, k: int,
             out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Token rows x [n, H] (bf16, fp16 or fp32) -> expert-sorted rows [n*k, H]:
    row row_sorted[t*k + j] is x[t]. The rows past the kept slots (an expert
    map drops some) are zero. `meta` as from route_metadata (row_sorted and
    offs are read)."""
    device = _need_rows(x, "x")
    n, H = x.shape
    _need_slots(meta, n * k, device)
    out = _out_rows(out, "out", (n * k, H), x)
    _run("moe_dispatch", device, x.data_ptr(), meta["row_sorted"].data_ptr(), _kept(meta), n, k,
         H, DTYPE[x.dtype], out.data_ptr())
    return out


def dispatch_backward(d_sorted: torch.Tensor, meta: dict, k: int,
                      out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Gradient of dispatch: d_sorted [n*k, H] -> d_x [n, H], each token the
    sum (fp32) of its kept slots' rows."""
    device = _need_rows(d_sorted, "d_sorted")
    N, H = d_sorted.shape
    if k < 1 or N % k:
        raise ValueError(f"d_sorted must have n*k rows, got {N} with k = {k}")
    n = N // k
    _need_slots(meta, N, device)
    out = _out_rows(out, "out", (n, H), d_sorted)
    _run("moe_dispatch_backward", device, d_sorted.data_ptr(), meta["row_sorted"].data_ptr(), n,
         k, H, DTYPE[d_sorted.dtype], out.data_ptr())
    return out


def combine_weighted(y_sorted: torch.Tensor, meta: dict, weights: torch.Tensor,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """Expert-sorted rows y_sorted [n*k, H] -> [n, H]: each token the sum
    (fp32) of its kept slots' rows times weights [n, k] (bf16 as route's
    topk_vals, or fp32)."""
    device = _need_rows(y_sorted, "y_sorted")
    _need_weights(weights, device)
    n, k = weights.shape
    N, H = y_sorted.shape
    if N != n * k:
        raise ValueError(f"y_sorted must have {n * k} rows, got {N}")
    _need_slots(meta, N, device)
    out = _out_rows(out, "out", (n, H), y_sorted)
    _run("moe_combine_weighted", device, y_sorted.data_ptr(), meta["row_sorted"].data_ptr(),
         weights.data_ptr(), DTYPE[weights.dtype], n, k, H, DTYPE[y_sorted.dtype],
         out.data_ptr())
    return out


def combine_weighted_backward(d_out: torch.Tensor, y_sorted: torch.Tensor, meta: dict,
                              weights: torch.Tensor):
    """Gradients of combine_weighted -> (d_sorted [n*k, H] of the rows' type,
    d_weights [n, k] fp32). Rows past the kept slots and the weights of
    dropped slots get zero."""
    device = _need_rows(d_out, "d_out")
    _need_weights(weights, device)
    n, k = weights.shape
    H = d_out.shape[1]
    if d_out.shape[0] != n:
        raise ValueError(f"d_out must have {n} rows, got {d_out.shape[0]}")
    _need_on(y_sorted, "y_sorted", d_out.dtype, device, (n * k, H))
    _need_slots(meta, n * k, device)
    d_sorted = d_out.new_empty((n * k, H))
    d_weights = torch.empty((n, k), dtype=torch.float32, device=d_out.device)
    _run("moe_combine_weighted_backward", device, d_out.data_ptr(), y_sorted.data_ptr(),
         meta["row_sorted"].data_ptr(), weights.data_ptr(), DTYPE[weights.dtype], _kept(meta), n,
         k, H, DTYPE[d_out.dtype], d_sorted.data_ptr(), d_weights.data_ptr())
    return d_sorted, d_weights


def route_backward(logits: torch.Tensor, topk_indx: torch.Tensor, d_vals: torch.Tensor,
                   gating: str = "softmax_topk") -> torch.Tensor:
    """Gradient of route's gate weights: d_vals fp32 [n, k] -> d_logits fp32 [n, E]."""
    _need(logits, "logits", torch.float32)
    if logits.dim() != 2:
        raise ValueError(f"logits must have shape [n, E], got {tuple(logits.shape)}")
    device = logits.get_device()
    n, E = logits.shape
    _need_on(topk_indx, "topk_indx", torch.int32, device)
    if topk_indx.dim() != 2 or topk_indx.shape[0] != n:
        raise ValueError(f"topk_indx must have shape [n, k], got {tuple(topk_indx.shape)}")
    k = topk_indx.shape[1]
    _need_on(d_vals, "d_vals", torch.float32, device, (n, k))
    d_logits = logits.new_empty((n, E))
    _run("moe_route_backward", device, logits.data_ptr(), topk_indx.data_ptr(),
         d_vals.data_ptr(), n, E, k, GATING[gating], d_logits.data_ptr())
    return d_logits


class Q4Weight:
    """4-bit weights as a checkpoint holds them: codes uint8 [R, C/2] (two E2M1
    codes per byte, the even column low) or [E, R, C/2], scales uint8
    [..., R, C/32] ("mxfp4": E8M0) or [..., R, C/16] ("nvfp4": E4M3, times
    matrix_scale fp32 [E] or [1]). The tensors are used where they lie; the
    handle keeps them alive and is theirs for good: other tensors take another
    handle."""

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, fmt: str,
                 matrix_scale: Optional[torch.Tensor] = None):
        if fmt not in Q4_FORMAT:
            raise ValueError(f"fmt must be one of {sorted(Q4_FORMAT)}, got {fmt!r}")
        _need(codes, "codes", torch.uint8)
        if codes.dim() not in (2, 3) or codes.shape[-1] == 0 or codes.shape[-1] % 16:
            raise ValueError("codes must have shape [R, C/2] or [E, R, C/2], C a multiple of 32")
        self.rows, self.cols = codes.shape[-2], 2 * codes.shape[-1]
        self.count = codes.shape[0] if codes.dim() == 3 else 1
        _need(scales, "scales", torch.uint8,
              (*codes.shape[:-1], self.cols // Q4_GROUP[fmt]))
        self.device = codes.get_device()
        _need_on(scales, "scales", torch.uint8, self.device,
                 (*codes.shape[:-1], self.cols // Q4_GROUP[fmt]))
        if matrix_scale is not None:
            _need_on(matrix_scale, "matrix_scale", torch.float32, self.device, (self.count,))
        self._codes, self._scales, self._matrix_scale, self._fmt = codes, scales, matrix_scale, fmt
        self._as_parameter_ = ctypes.byref(Q4Matrix(
            codes.data_ptr(), scales.data_ptr(),
            None if matrix_scale is None else matrix_scale.data_ptr(), Q4_FORMAT[fmt]))

    codes = property(lambda self: self._codes)
    scales = property(lambda self: self._scales)
    matrix_scale = property(lambda self: self._matrix_scale)
    fmt = property(lambda self: self._fmt)


def _need_q4(w: Q4Weight, name: str, device: int) -> None:
    if not isinstance(w, Q4Weight):
        raise ValueError(f"{name} must be a Q4Weight")
    if w.device != device:
        raise ValueError(f"{name} is on cuda:{w.device}, not on cuda:{device}")


def _need_q4_x(x: torch.Tensor) -> int:
    device = _need_rows(x, "x")
    if x.dtype is torch.float32:
        raise ValueError("x must be bfloat16 or float16")
    return device


def linear_q4(x: torch.Tensor, w: Q4Weight, out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """x [n, C] (bf16 or fp16) times one 4-bit matrix [R, C] -> [n, R]."""
    device = _need_q4_x(x)
    _need_q4(w, "w", device)
    n, C = x.shape
    if w.count != 1 or w.cols != C:
        raise ValueError(f"w must be one matrix of {C} columns, got {tuple(w.codes.shape)} codes")
    out = _out_rows(out, "out", (n, w.rows), x)
    _run("moe_linear_q4", device, x.data_ptr(), w, n, w.rows, C, DTYPE[x.dtype], out.data_ptr())
    return out


def workspace_q4_size(n: int, E: int, k: int, H: int, I: int) -> int:
    return int(lib().moe_q4_workspace_size(n, E, k, H, I))


def workspace_q4(n: int, E: int, k: int, H: int, I: int,
                 device: Optional[torch.device] = None) -> torch.Tensor:
    """Allocate and initialise a workspace for grouped_ffn_q4 and forward_q4."""
    size = workspace_q4_size(n, E, k, H, I)
    if size == 0:
        raise ValueError("invalid sizes for moe_q4_workspace_size")
    ws = torch.empty(size, dtype=torch.uint8,
                     device=torch.device("cuda") if device is None else torch.device(device))
    with torch.cuda.device(ws.device):
        _check(lib().moe_workspace_init(_ptr(ws), size, _stream(ws.device)), "moe_workspace_init")
    return ws


def _q4_experts(w13: Q4Weight, w2: Q4Weight, E: int, H: int, device: int,
                params: MoeParams) -> int:
    """Checks the experts' matrices against each other; returns I."""
    _need_q4(w13, "w13", device)
    _need_q4(w2, "w2", device)
    I = w2.cols
    rows = I if params.activation == ACT["relu2"] else 2 * I
    if (w13.count, w13.rows, w13.cols) != (E, rows, H):
        raise ValueError(f"w13 must be {E} matrices of {rows} x {H}, got "
                         f"{(w13.count, w13.rows, w13.cols)}")
    if (w2.count, w2.rows) != (E, H):
        raise ValueError(f"w2 must be {E} matrices of {H} rows, got {(w2.count, w2.rows)}")
    return I


def grouped_ffn_q4(x: torch.Tensor, meta: dict, w13: Q4Weight, w2: Q4Weight, k: int,
                   ws: torch.Tensor, params: MoeParams,
                   out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The experts of a decode step with 4-bit weights: x [n, H] (bf16 or
    fp16) -> their outputs in expert-sorted order [n*k, H], without gate
    weights (combine_weighted applies them); rows past the kept slots are
    zero. `ws` from workspace_q4."""
    device = _need_q4_x(x)
    n, H = x.shape
    E = w13.count if isinstance(w13, Q4Weight) else 0
    I = _q4_experts(w13, w2, E, H, device, params)
    offs, col_sorted = meta["offs"], meta["col_sorted"]
    _need_on(offs, "offs", torch.int32, device, (E + 1,))
    _need_on(col_sorted, "col_sorted", torch.int32, device, (n * k,))
    _need_on(ws, "ws", torch.uint8, device)
    out = _out_rows(out, "out", (n * k, H), x)
    m = RoutingMeta(None, offs.data_ptr(), col_sorted.data_ptr(), None, None)
    _run("moe_grouped_ffn_q4", device, x.data_ptr(), ctypes.byref(m), w13, w2, n, E, k, H, I,
         ctypes.byref(params), DTYPE[x.dtype], out.data_ptr(), ws.data_ptr(), ws.numel())
    return out


def forward_q4(x: torch.Tensor, logits: torch.Tensor, w13: Q4Weight, w2: Q4Weight, k: int,
               params: MoeParams, ws: torch.Tensor, out: Optional[torch.Tensor] = None,
               topk: Optional[tuple] = None, meta: Optional[dict] = None) -> torch.Tensor:
    """forward() with 4-bit experts: route_metadata, grouped_ffn_q4 and
    combine_weighted in one library call. x and out bf16 or fp16, `ws` from
    workspace_q4."""
    device = _need_q4_x(x)
    n, H = x.shape
    _need_on(logits, "logits", torch.float32, device)
    if logits.dim() != 2 or logits.shape[0] != n:
        raise ValueError(f"logits must have shape [{n}, E], got {tuple(logits.shape)}")
    E = logits.shape[1]
    E_w = params.n_local_experts if params.expert_map else E  # experts held in w13 / w2
    I = _q4_experts(w13, w2, E_w, H, device, params)
    _need_on(ws, "ws", torch.uint8, device)
    out = _out_rows(out, "out", (n, H), x)
    indx = vals = None
    if topk is not None:
        indx, vals = topk
        _need_on(indx, "topk_indx", torch.int32, device, (n, k))
        _need_on(vals, "topk_vals", torch.bfloat16, device, (n, k))
    mstruct = None
    if meta is not None:
        for name, dtype, size in (("col_sum", torch.int32, E_w), ("offs", torch.int32, E_w + 1),
                                  ("col_sorted", torch.int32, n * k),
                                  ("row_sorted", torch.int32, n * k),
                                  ("gate_scal", torch.bfloat16, n * k)):
            _need_on(meta[name], name, dtype, device, (size,))
        mstruct = ctypes.byref(_meta_struct(meta))
    _run("moe_forward_q4", device, x.data_ptr(), logits.data_ptr(), w13, w2, n, E, k, H, I,
         ctypes.byref(params), DTYPE[x.dtype], out.data_ptr(), _ptr(indx), _ptr(vals), mstruct,
         ws.data_ptr(), ws.numel())
    return out


class Mx8:
    """MXFP8 rows: codes float8_e4m3fn [rows, C] and scales uint8 [rows, C/32]
    (E8M0), C a multiple of 32. The tensors are used where they lie at each
    call; the handle keeps them alive and is theirs for good: other tensors
    take another handle."""

    __slots__ = ("_codes", "_scales", "_rows", "device", "shape")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor):
        self.device = codes.get_device() if isinstance(codes, torch.Tensor) else -1
        _need_on(codes, "codes", torch.float8_e4m3fn, self.device)
        if codes.dim() != 2 or codes.shape[1] == 0 or codes.shape[1] % 32:
            raise ValueError(f"codes must have shape [rows, C], C a multiple of 32, got "
                             f"{tuple(codes.shape)}")
        self.shape = codes.shape
        _need_on(scales, "scales", torch.uint8, self.device, (self.shape[0], self.shape[1] // 32))
        self._codes, self._scales, self._rows = codes, scales, Mx8Rows()

    @property
    def codes(self) -> torch.Tensor:
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        return self._scales

    def _argument(self):
        """The library's argument, with the tensors' addresses as they are now (a
        tensor can be given other memory, or another shape, behind the handle)."""
        c, s, shape = self._codes, self._scales, self.shape
        if not (c.shape == shape and s.shape == (shape[0], shape[1] // 32)
                and c.is_contiguous() and s.is_contiguous()
                and c.get_device() == s.get_device() == self.device):
            raise ValueError("codes or scales are no longer as they were when the handle was made")
        rows = self._rows
        rows.codes, rows.scales = c.data_ptr(), s.data_ptr()
        return ctypes.byref(rows)


def _empty_mx8(rows: int, cols: int, like: torch.Tensor, device: int) -> Mx8:
    if cols % 32:
        raise ValueError(f"8-bit rows need a multiple of 32 columns, got {cols}")
    m = Mx8.__new__(Mx8)
    on = like.device
    m._codes = torch.empty((rows, cols), dtype=torch.float8_e4m3fn, device=on)
    m._scales = torch.empty((rows, cols // 32), dtype=torch.uint8, device=on)
    m._rows = Mx8Rows(m._codes.data_ptr(), m._scales.data_ptr())
    m.device, m.shape = device, m._codes.shape
    return m


def _out_like(out: Optional[torch.Tensor], name: str, like: torch.Tensor) -> torch.Tensor:
    """`out`, or a new tensor, of like's shape and type (empty_like costs the
    host 2 us less than new_empty)."""
    if out is None:
        return torch.empty_like(like)
    _need_on(out, name, like.dtype, like.get_device(), like.shape)
    return out


def _need_rows16(t: torch.Tensor, name: str) -> int:
    device = _need_rows(t, name)
    if t.dtype is torch.float32:
        raise ValueError(f"{name} must be bfloat16 or float16")
    return device


def _need_vector(t: torch.Tensor, name: str, dtypes: tuple, device: int, size: int) -> int:
    """A [size] vector of one of the types; its address."""
    if not isinstance(t, torch.Tensor) or t.dtype not in dtypes:
        raise ValueError(f"{name} must be a tensor of {' or '.join(map(str, dtypes))}")
    _need_on(t, name, t.dtype, device, (size,))
    return t.data_ptr()


def _need_status(status: Optional[torch.Tensor], device: int):
    """Address of the optional status word (int32 [1], zeroed by the caller)."""
    if status is None:
        return None
    _need_on(status, "status", torch.int32, device, (1,))
    return status.data_ptr()


def _scratch(ws: Optional[torch.Tensor], size: int, like: torch.Tensor, device: int):
    """(workspace tensor or None, address, bytes): the caller's, or a new one."""
    if ws is None:
        if size == 0:
            return None, None, 0
        ws = torch.empty(size, dtype=torch.uint8, device=like.device)
    else:
        _need_on(ws, "ws", torch.uint8, device)
    return ws, ws.data_ptr(), ws.numel()


def _weight_vector(weight: torch.Tensor, dt: torch.dtype, device: int, H: int):
    """(address, type) of a norm's weights: [H] of the rows' type or fp32."""
    if (isinstance(weight, torch.Tensor) and (weight.dtype is dt or weight.dtype is torch.float32)
            and weight.dim() == 1 and weight.numel() == H and weight.is_contiguous()
            and weight.get_device() == device):
        return weight.data_ptr(), DTYPE[weight.dtype]
    return _need_vector(weight, "weight", (dt, torch.float32), device, H), DTYPE[weight.dtype]


def rms_norm(x: torch.Tensor, weight: Optional[torch.Tensor], eps: float = 1e-5,
             residual: Optional[torch.Tensor] = None, mx8: bool = False, out=None,
             sum_out: Optional[torch.Tensor] = None):
    """Root-mean-square norm of the rows x [n, H] (bf16, fp16 or fp32) times
    weight [H] (of x's type or fp32; None: ones). With a residual [n, H] the
    norm is of s = x + residual, rounded to x's type, and the result is (y, s).
    mx8: y is Mx8 rows (H a multiple of 32). out, sum_out: where y and s go."""
    device = _need_rows(x, "x")
    n, H = shape = x.shape
    dt = x.dtype
    dtype = w_dtype = DTYPE[dt]
    w = r = t = total = None
    if weight is not None:
        w, w_dtype = _weight_vector(weight, dt, device, H)
    if residual is not None:
        _need_on(residual, "residual", dt, device, shape)
        r = residual.data_ptr()
        total = torch.empty_like(x) if sum_out is None else _out_like(sum_out, "sum_out", x)
        t = total.data_ptr()
    elif sum_out is not None:
        raise ValueError("sum_out needs a residual")
    if mx8:
        if out is None:
            y = _empty_mx8(n, H, x, device)
            y8 = ctypes.byref(y._rows)
        else:
            y = out
            _need_mx8(y, "out", device, shape)
            y8 = y._argument()
        _run("moe_rms_norm", device, x.data_ptr(), r, w, w_dtype, n, H, dtype, eps, None, y8, t)
    else:
        y = torch.empty_like(x) if out is None else _out_like(out, "out", x)
        _run("moe_rms_norm", device, x.data_ptr(), r, w, w_dtype, n, H, dtype, eps, y.data_ptr(),
             None, t)
    return y if residual is None else (y, total)


def _need_mx8(m: Mx8, name: str, device: int, shape=None) -> None:
    if not isinstance(m, Mx8):
        raise ValueError(f"{name} must be Mx8 rows")
    if m.device != device:
        raise ValueError(f"{name} is on cuda:{m.device}, not on cuda:{device}")
    if shape is not None and m.shape != shape:
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(m.shape)}")


def rms_norm_backward(d_y: torch.Tensor, x: torch.Tensor, weight: Optional[torch.Tensor],
                      eps: float = 1e-5, d_sum: Optional[torch.Tensor] = None,
                      ws: Optional[torch.Tensor] = None):
    """Gradients of rms_norm -> (d_x [n, H], d_weight [H] of weight's type, or
    None without a weight). x is what was normalised (the sum, where there was
    a residual; d_x is then the gradient of x and of the residual alike), d_sum the
    gradient that reaches the sum from elsewhere, added to d_x. ws: scratch
    (rms_norm_backward_workspace_size), allocated where it is None."""
    device = _need_rows(x, "x")
    n, H = x.shape
    _need_on(d_y, "d_y", x.dtype, device, (n, H))
    if d_sum is not None:
        _need_on(d_sum, "d_sum", x.dtype, device, (n, H))
    w_dtype, w, d_weight, size = DTYPE[x.dtype], None, None, 0
    if weight is not None:
        w, w_dtype = _weight_vector(weight, x.dtype, device, H)
        d_weight = torch.empty_like(weight)
        size = rms_norm_backward_workspace_size(n, H)
    d_x = torch.empty_like(x)
    ws, p, size = _scratch(ws, size, x, device)
    _run("moe_rms_norm_backward", device, d_y.data_ptr(), x.data_ptr(), w, w_dtype,
         None if d_sum is None else d_sum.data_ptr(), n, H, DTYPE[x.dtype], eps, d_x.data_ptr(),
         None if d_weight is None else d_weight.data_ptr(), p, size)
    return d_x, d_weight


@functools.lru_cache(maxsize=4096)
def rms_norm_backward_workspace_size(n: int, H: int) -> int:
    return int((_LIB or lib()).moe_rms_norm_backward_workspace_size(n, H))


@functools.lru_cache(maxsize=4096)
def linear_workspace_size(n: int, R: int, C: int, mx8: bool = False) -> int:
    """Bytes of scratch for linear; mx8: with Mx8 operands."""
    return int((_LIB or lib()).moe_linear_workspace_size(n, R, C, mx8))


@functools.lru_cache(maxsize=4096)
def linear_backward_workspace_size(n: int, R: int, C: int, act: str = "none") -> int:
    return int((_LIB or lib()).moe_linear_backward_workspace_size(n, R, C, LINEAR_ACT[act]))


@functools.lru_cache(maxsize=4096)
def gated_linear_workspace_size(n: int, H: int, I: int, mx8: bool = False,
                                h_mx8: bool = False) -> int:
    """Bytes of scratch for gated_linear; mx8 / h_mx8: with Mx8 operands / results."""
    return int((_LIB or lib()).moe_gated_linear_workspace_size(n, H, I, mx8, h_mx8))


@functools.lru_cache(maxsize=4096)
def gated_linear_backward_workspace_size(n: int, H: int, I: int) -> int:
    return int((_LIB or lib()).moe_gated_linear_backward_workspace_size(n, H, I))


def _need_act(act: str) -> int:
    act_id = LINEAR_ACT.get(act)
    if act_id is None:
        raise ValueError(f"act must be one of {sorted(LINEAR_ACT)}, got {act!r}")
    return act_id


def _product_operands(x, w, w_name: str, dtype):
    """(device, rows, features, out features, output type) of x and w, both
    16-bit tensors of one type or both Mx8. One expression checks the common
    case; what it refuses is then named."""
    if type(x) is Mx8:
        device = x.device
        _need_mx8(w, w_name, device)
        if w.shape[1] != x.shape[1]:
            raise ValueError(f"{w_name} must have {x.shape[1]} columns, got {tuple(w.shape)}")
        dtype = torch.bfloat16 if dtype is None else dtype
        if dtype not in (torch.bfloat16, torch.float16):
            raise ValueError("dtype must be torch.bfloat16 or torch.float16")
        return device, x.shape[0], x.shape[1], w.shape[0], dtype
    if isinstance(x, torch.Tensor) and isinstance(w, torch.Tensor) and x.dim() == 2 == w.dim():
        dt, device = x.dtype, x.get_device()
        n, C = x.shape
        R, columns = w.shape
        if ((dt is torch.bfloat16 or dt is torch.float16) and w.dtype is dt and columns == C > 0
                and w.get_device() == device >= 0 and x.is_contiguous() and w.is_contiguous()
                and (dtype is None or dtype is dt)):
            return device, n, C, R, dt
    device = _need_rows16(x, "x")
    if dtype is not None and dtype is not x.dtype:
        raise ValueError(f"dtype is x's, {x.dtype}, unless x is Mx8 rows")
    _need_on(w, w_name, x.dtype, device)
    raise ValueError(f"{w_name} must have shape [rows, {x.shape[1]}], got {tuple(w.shape)}")


def linear(x, w, bias: Optional[torch.Tensor] = None, act: str = "none",
           residual: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
           ws: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
           status: Optional[torch.Tensor] = None) -> torch.Tensor:
    """act(x w^T + bias) + residual: x [n, C] and w [R, C] bf16 or fp16, or
    both Mx8 rows (dtype: that of the result then, bf16 by default). act:
    "none", "silu", "gelu" or "relu2"; bias [R], residual [n, R]. ws: scratch
    (linear_workspace_size), allocated where it is None."""
    act_id = _need_act(act)
    device, n, C, R, dtype = _product_operands(x, w, "w", dtype)
    if type(x) is Mx8:
        name, like, xp, wp = "moe_linear_mx8", x.codes, x._argument(), w._argument()
    else:
        name, like, xp, wp = "moe_linear", x, x.data_ptr(), w.data_ptr()
    b = None if bias is None else _need_vector(bias, "bias", (dtype,), device, R)
    if residual is not None:
        _need_on(residual, "residual", dtype, device, (n, R))
        residual = residual.data_ptr()
    if out is None:
        out = torch.empty((n, R), dtype=dtype, device=like.device)
    else:
        _need_on(out, "out", dtype, device, (n, R))
    size = linear_workspace_size(n, R, C, like is not x)
    p = None
    if size or ws is not None:
        ws, p, size = _scratch(ws, size, like, device)
    if status is not None:
        status = _need_status(status, device)
    _run(name, device, xp, wp, b, residual, n, R, C, DTYPE[dtype], act_id, out.data_ptr(), p, size,
         status)
    return out


def linear_backward(d_y: torch.Tensor, x: torch.Tensor, w: torch.Tensor,
                    bias: Optional[torch.Tensor] = None, act: str = "none",
                    ws: Optional[torch.Tensor] = None, status: Optional[torch.Tensor] = None):
    """Gradients of linear (16-bit operands) for d_y [n, R] -> (d_x [n, C],
    d_w [R, C], d_bias [R] or None without a bias). The residual's gradient is
    d_y. R a multiple of 8. ws: scratch (linear_backward_workspace_size),
    allocated where it is None."""
    act_id = _need_act(act)
    device, n, C, R, dtype = _product_operands(x, w, "w", None)
    _need_on(d_y, "d_y", dtype, device, (n, R))
    b = None if bias is None else _need_vector(bias, "bias", (dtype,), device, R)
    d_x, d_w = torch.empty_like(x), torch.empty_like(w)
    d_bias = None if bias is None else torch.empty_like(bias)
    ws, p, size = _scratch(ws, linear_backward_workspace_size(n, R, C, act), x, device)
    _run("moe_linear_backward", device, d_y.data_ptr(), x.data_ptr(), w.data_ptr(), b, n, R, C,
         DTYPE[dtype], act_id, d_x.data_ptr(), d_w.data_ptr(),
         None if d_bias is None else d_bias.data_ptr(), p, size, _need_status(status, device))
    return d_x, d_w, d_bias


def gated_linear(x, w13, params: MoeParams, out=None, mx8: bool = False,
                 ws: Optional[torch.Tensor] = None, dtype: Optional[torch.dtype] = None,
                 status: Optional[torch.Tensor] = None):
    """The gated activation of (gate, up) = x w13^T: x [n, H] and w13 [2I, H]
    (rows in params' layout) bf16 or fp16, or both Mx8 rows -> h [n, I] of x's
    type (Mx8 operands: of `dtype`, bf16 by default), or Mx8 rows with mx8 (I a
    multiple of 32). params: make_params' activation ("swiglu" or
    "swiglu_oai"), layout and limits. ws: scratch
    (gated_linear_workspace_size), allocated where it is None."""
    device, n, H, rows, dtype = _product_operands(x, w13, "w13", dtype)
    if rows % 2:
        raise ValueError(f"w13 must have an even number of rows, got {rows}")
    I = rows // 2
    if type(x) is Mx8:
        name, like, xp, wp = "moe_gated_linear_mx8", x.codes, x._argument(), w13._argument()
    else:
        name, like, xp, wp = "moe_gated_linear", x, x.data_ptr(), w13.data_ptr()
    if mx8:
        if out is None:
            out = _empty_mx8(n, I, like, device)
            h8 = ctypes.byref(out._rows)
        else:
            _need_mx8(out, "out", device, (n, I))
            h8 = out._argument()
        hp = None
    else:
        if out is None:
            out = torch.empty((n, I), dtype=dtype, device=like.device)
        else:
            _need_on(out, "out", dtype, device, (n, I))
        hp, h8 = out.data_ptr(), None
    size = gated_linear_workspace_size(n, H, I, like is not x, mx8)
    p = None
    if size or ws is not None:
        ws, p, size = _scratch(ws, size, like, device)
    if status is not None:
        status = _need_status(status, device)
    _run(name, device, xp, wp, n, H, I, ctypes.byref(params), DTYPE[dtype], hp, h8, p, size, status)
    return out


def gated_linear_backward(d_h: torch.Tensor, x: torch.Tensor, w13: torch.Tensor,
                          params: MoeParams, ws: Optional[torch.Tensor] = None,
                          status: Optional[torch.Tensor] = None):
    """Gradients of gated_linear (16-bit operands) for d_h [n, I] -> (d_x
    [n, H], d_w13 [2I, H]). ws: scratch (gated_linear_backward_workspace_size),
    allocated where it is None."""
    device, n, H, rows, dtype = _product_operands(x, w13, "w13", None)
    if rows % 2:
        raise ValueError(f"w13 must have an even number of rows, got {rows}")
    I = rows // 2
    _need_on(d_h, "d_h", dtype, device, (n, I))
    d_x, d_w13 = torch.empty_like(x), torch.empty_like(w13)
    ws, p, size = _scratch(ws, gated_linear_backward_workspace_size(n, H, I), x, device)
    _run("moe_gated_linear_backward", device, d_h.data_ptr(), x.data_ptr(), w13.data_ptr(), n, H,
         I, ctypes.byref(params), DTYPE[dtype], d_x.data_ptr(), d_w13.data_ptr(), p, size,
         _need_status(status, device))
    return d_x, d_w13


STAGES = ("route", "metadata", "gather", "ffn1", "ffn2", "combine")


def forward_timed(x: torch.Tensor, logits: torch.Tensor, w13: torch.Tensor, w2: torch.Tensor,
                  k: int, params: MoeParams, ws: torch.Tensor, events: list,
                  out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """forward() that records len(STAGES) + 1 torch.cuda.Event objects between
    the stage kernels (events[i] before stage i, the last after the end)."""
    n, H = x.shape
    E = logits.shape[1]
    I = _intermediate(w13, params)
    if out is None:
        out = torch.empty((n, H), dtype=torch.bfloat16, device=x.device)
    if len(events) != len(STAGES) + 1:
        raise ValueError("need len(STAGES) + 1 events")
    for e in events:
        if not e.cuda_event:  # torch creates the CUDA event on its first record
            e.record()
    arr = (ctypes.c_void_p * len(events))(*[ctypes.c_void_p(e.cuda_event) for e in events])
    _check(lib().moe_forward_timed(_ptr(x), _ptr(logits), _ptr(w13), _ptr(w2), n, E, k, H, I,
                                   ctypes.byref(params), _ptr(out), None, None, None, _ptr(ws),
                                   ws.numel(), arr, len(events), _stream(x.device)),
           "moe_forward_timed")
    return out


def forward_launch_count(n: int, E: int, k: int, H: int, I: int) -> int:
    """Kernels one moe_forward enqueues for these sizes (-1: invalid sizes)."""
    return int(lib().moe_forward_launch_count(n, E, k, H, I))


def ffn_plan(n: int, E: int, k: int, H: int, I: int, params: MoeParams) -> dict:
    """How the two expert contractions are tiled for these sizes (no launch):
    token rows per tile of each, whether each runs on CTA pairs, whether the
    decode tiling applies, and whether both run in one launch."""
    plan = (ctypes.c_int32 * 6)()
    _check(lib().moe_ffn_plan(n, E, k, H, I, ctypes.byref(params), plan), "moe_ffn_plan")
    return {"token_tile_w13": plan[0], "token_tile_w2": plan[1], "pair_w13": bool(plan[2]),
            "pair_w2": bool(plan[3]), "decode": bool(plan[4]), "fused": bool(plan[5])}


def read_status(ws: Optional[torch.Tensor] = None, reset: bool = False) -> int:
    """DEBUG: synchronises and returns the device status word (0 = OK) of a
    workspace or, without one, of the current device: the one where linear,
    gated_linear and their gradients record a wait that gave up when they were
    given no `status`."""
    if ws is None:
        stream = torch._C._cuda_getCurrentRawStream(torch.cuda.current_device())
        return int(lib().moe_read_dense_status(int(reset), stream))
    return int(lib().moe_read_status(_ptr(ws), ws.numel(), int(reset), _stream(ws.device)))


def selftest_wait_timeout(ws: torch.Tensor, timeout_ns: int) -> None:
    _check(lib().moe_selftest_wait_timeout(_ptr(ws), ws.numel(), int(timeout_ns),
                                           _stream(ws.device)), "moe_selftest_wait_timeout")
