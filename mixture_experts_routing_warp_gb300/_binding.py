"""ctypes binding over the C ABI in include/moe.h (argument marshalling only).

Every stage runs in the CUDA library libmoe_gb300.so; this module checks
tensor devices / dtypes / shapes, allocates outputs with PyTorch, passes
`data_ptr()`s and the current CUDA stream, and turns a non-zero moe_status
into an exception. There is no fallback: if the library is missing, every
call raises.
"""
from __future__ import annotations

import ctypes
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


_LIB = None

# name -> (restype, argtypes)
_P, _I64, _I32, _SZ, _U64 = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_size_t,
                             ctypes.c_uint64)
_PP = ctypes.POINTER(MoeParams)
_PM = ctypes.POINTER(RoutingMeta)
_PQ = ctypes.POINTER(Q4Matrix)
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
    "moe_read_status": (_I32, [_P, _SZ, _I32, _P]),
    "moe_selftest_wait_timeout": (_I32, [_P, _SZ, _U64, _P]),
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
    if device == torch.cuda.current_device():
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
    handle keeps them alive."""

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
        self.codes, self.scales, self.matrix_scale, self.fmt = codes, scales, matrix_scale, fmt
        self._as_parameter_ = ctypes.byref(Q4Matrix(
            codes.data_ptr(), scales.data_ptr(),
            None if matrix_scale is None else matrix_scale.data_ptr(), Q4_FORMAT[fmt]))


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


def read_status(ws: torch.Tensor, reset: bool = False) -> int:
    """DEBUG: synchronises and returns the device status word (0 = OK)."""
    return int(lib().moe_read_status(_ptr(ws), ws.numel(), int(reset), _stream(ws.device)))


def selftest_wait_timeout(ws: torch.Tensor, timeout_ns: int) -> None:
    _check(lib().moe_selftest_wait_timeout(_ptr(ws), ws.numel(), int(timeout_ns),
                                           _stream(ws.device)), "moe_selftest_wait_timeout")
