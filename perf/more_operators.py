"""The dense blocks beside the expert layer, as cases to time and to compare.

A transformer block around the expert layer, or its shared expert, is
    s, y = rms_norm(x, weight, residual)      the norm with the residual's addition
    h    = gated_linear(y, w13)               both projections, the activation, the product
    out  = linear(h, w2, bias, residual=s)    a product with its epilogue
and its gradients. Each operator has its plain form here in elementary torch
operations and the call that a user makes of
`mixture_experts_routing_warp_gb300`. Rows are bf16 or fp16 (the norm: fp32
too) or, without gradients, MXFP8: E4M3 codes with one E8M0 scale per 32.
"""
import math

import torch

own = False

_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4, "mx8": 1 + 1 / 32}
_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_EPS = 1e-5
_ALPHA, _BETA, _LIMIT = 1.702, 1.0, 7.0   # SwiGLU-OAI


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # the norm in front of a layer, a decode step of 8 sequences: latency
        dict(name="norm_n8_h2880", op="norm", n=8, H=2880, dtype="bf16", residual=True, out="same"),
        # the largest prefill, written in 8 bits for the product that follows
        dict(name="norm_n16384_h2880_mx8", op="norm", n=16384, H=2880, dtype="bf16",
             residual=True, out="mx8"),
        # its gradients in a training step, the residual stream's gradient added
        dict(name="norm_grad_n8192_h2880", op="norm_grad", n=8192, H=2880, dtype="bf16",
             residual=True),
        # float rows of an odd length
        dict(name="norm_grad_n517_h1001_fp32", op="norm_grad", n=517, H=1001, dtype="fp32",
             residual=False),
        # the projection back to the residual stream, one new token
        dict(name="linear_n1_2880x2880", op="linear", n=1, R=2880, C=2880, dtype="bf16",
             bias=False, act="none", residual=True),
        # the same for a prompt, with a bias
        dict(name="linear_n8192_2880x2880", op="linear", n=8192, R=2880, C=2880, dtype="bf16",
             bias=True, act="none", residual=True),
        # 8-bit rows and weights, an odd number of tokens
        dict(name="linear_n2047_5760x2880_mx8", op="linear", n=2047, R=5760, C=2880, dtype="mx8",
             bias=True, act="none", residual=False),
        # gradients of a small projection with an activation (MiniMind's sizes)
        dict(name="linear_grad_n4096_512x1408_fp16", op="linear_grad", n=4096, R=512, C=1408,
             dtype="fp16", bias=True, act="silu"),
        # a shared expert beside the routed ones: 8 sequences, one token each
        dict(name="gated_n8_2880", op="gated", n=8, H=2880, I=2880, dtype="bf16",
             act="swiglu_oai", layout="interleaved", out="same"),
        # the same for a prompt, in 8 bits from the norm to the next product
        dict(name="gated_n8192_2880_mx8", op="gated", n=8192, H=2880, I=2880, dtype="mx8",
             act="swiglu_oai", layout="interleaved", out="mx8"),
        # a dense block of MiniMind's sizes, forward
        dict(name="gated_n4096_512x1408", op="gated", n=4096, H=512, I=1408, dtype="bf16",
             act="swiglu", layout="packed", out="same"),
        # gradients of the shared expert in a training step: the largest case
        dict(name="gated_grad_n8192_2880", op="gated_grad", n=8192, H=2880, I=2880, dtype="bf16",
             act="swiglu", layout="packed"),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    done = [work(c) for c in listed()]
    top = {k: max(w[k] for w in done) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["norm", "norm_grad", "linear", "linear", "linear_grad", "gated", "gated",
                         "gated_grad"])
        n = _log_int(rng, 1, 16384)
        if op in ("norm", "norm_grad"):
            case = dict(op=op, n=n, H=_log_int(rng, 16, 8192),
                        dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                        residual=rng.random() < 0.5)
            if op == "norm":
                case["out"] = "mx8" if rng.random() < 0.4 else "same"
            if case.get("out") == "mx8":
                case["H"] = 32 * _log_int(rng, 1, 256)
            elif rng.random() < 0.5:
                case["H"] = 8 * _log_int(rng, 2, 1024)
        elif op == "linear":
            dtype = rng.choice(["bf16", "fp16", "mx8"])
            case = dict(op=op, n=n, R=_log_int(rng, 1, 8192),
                        C=(32 if dtype == "mx8" else 8) * _log_int(rng, 8, 256), dtype=dtype,
                        bias=rng.random() < 0.5, act=rng.choice(["none", "silu", "gelu", "relu2"]),
                        residual=rng.random() < 0.5)
        elif op == "linear_grad":
            case = dict(op=op, n=n, R=8 * _log_int(rng, 8, 720), C=8 * _log_int(rng, 8, 720),
                        dtype=rng.choice(["bf16", "fp16"]), bias=rng.random() < 0.5,
                        act=rng.choice(["none", "silu", "gelu", "relu2"]))
        else:
            dtype = rng.choice(["bf16", "fp16", "mx8"]) if op == "gated" else \
                rng.choice(["bf16", "fp16"])
            case = dict(op=op, n=n, H=8 * _log_int(rng, 8, 512), I=8 * _log_int(rng, 8, 512),
                        dtype=dtype, act=rng.choice(["swiglu", "swiglu_oai"]),
                        layout=rng.choice(["packed", "interleaved"]))
            if dtype == "mx8":
                case["H"] = 32 * _log_int(rng, 2, 128)
            if op == "gated":
                case["out"] = "same"
                if rng.random() < 0.4:
                    case.update(out="mx8", I=32 * _log_int(rng, 2, 128))
        w = work(case)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            return case


def work(case):
    op, n, s = case["op"], case["n"], _BYTES[case["dtype"]]
    o = 2 if case["dtype"] == "mx8" else s            # 8-bit products come out as bf16
    if op == "norm":
        H, y = case["H"], _BYTES["mx8"] if case["out"] == "mx8" else s
        return {"bytes": int(n * H * (s + y + (2 * s if case["residual"] else 0)) + H * s),
                "flops": 4 * n * H}
    if op == "norm_grad":
        H = case["H"]
        return {"bytes": n * H * s * (4 if case["residual"] else 3) + 2 * H * s,
                "flops": 9 * n * H}
    if op == "linear":
        R, C = case["R"], case["C"]
        return {"bytes": int(n * C * s + R * C * s + n * R * o * (2 if case["residual"] else 1) +
                             (R * o if case["bias"] else 0)),
                "flops": 2 * n * R * C}
    if op == "linear_grad":
        R, C = case["R"], case["C"]
        products = 2 if case["act"] == "none" else 3   # an activation needs its argument again
        return {"bytes": n * R * s + 2 * n * C * s + 2 * R * C * s +
                (2 * R * s if case["bias"] else 0),
                "flops": products * 2 * n * R * C}
    H, I = case["H"], case["I"]
    if op == "gated":
        h = _BYTES["mx8"] if case["out"] == "mx8" else o
        return {"bytes": int(n * H * s + 2 * I * H * s + n * I * h), "flops": 4 * n * I * H}
    return {"bytes": n * I * s + 2 * n * H * s + 4 * I * H * s, "flops": 12 * n * I * H}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x0DE5E000 + seed)
    return g


def _randn(g, *shape):
    return torch.randn(*shape, generator=g, device="cuda")


def _scale_exponent(v):
    """[rows, C/32] exponents: the least power of two under which every value
    of a group of 32 is at most 448, E4M3's largest (2^-127 at the least)."""
    m, e = torch.frexp(v.view(v.shape[0], -1, 32).abs().amax(dim=2))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    return torch.where(m == 0, torch.full_like(e, -127), e).clamp_min(-127)


def _quantise(v):
    """float32 rows [rows, C] -> E4M3 codes and E8M0 scale bytes."""
    e = _scale_exponent(v)
    u = torch.ldexp(v.view(v.shape[0], -1, 32), -e[:, :, None])
    return u.view_as(v).to(torch.float8_e4m3fn), (e + 127).to(torch.uint8)


def _operand(v, dtype):
    if dtype != "mx8":
        return v.to(_DTYPE[dtype])
    codes, scales = _quantise(v)
    return {"codes": codes, "scales": scales}


def prepare(case, seed):
    g = _gen(seed)
    op, n, dtype = case["op"], case["n"], case["dtype"]
    st = {"case": case}
    row = torch.bfloat16 if dtype == "mx8" else _DTYPE[dtype]
    if op in ("norm", "norm_grad"):
        H = case["H"]
        # rows of different magnitude, as a residual stream has
        x = _randn(g, n, H) * torch.exp(0.5 * _randn(g, n, 1))
        st["x"] = x.to(row)
        st["weight"] = (1.0 + 0.1 * _randn(g, H)).to(row)
        if case["residual"]:
            st["residual" if op == "norm" else "d_sum"] = _randn(g, n, H).to(row)
        if op == "norm_grad":
            st["d_y"] = _randn(g, n, H).to(row)
    elif op in ("linear", "linear_grad"):
        R, C = case["R"], case["C"]
        st["x"] = _operand(_randn(g, n, C), dtype)
        st["w"] = _operand(_randn(g, R, C) * C ** -0.5, dtype)
        if case["bias"]:
            st["bias"] = _randn(g, R).to(row)
        if op == "linear" and case["residual"]:
            st["residual"] = _randn(g, n, R).to(row)
        if op == "linear_grad":
            st["d_y"] = _randn(g, n, R).to(row)
    else:
        H, I = case["H"], case["I"]
        st["x"] = _operand(_randn(g, n, H), dtype)
        st["w13"] = _operand(_randn(g, 2 * I, H) * H ** -0.5, dtype)
        if op == "gated_grad":
            st["d_h"] = _randn(g, n, I).to(row)
    return st


# ------------------------------------------------------------- plain forms --

def _f32(v):
    """float32 of a 16-bit tensor, or of 8-bit codes with their scales."""
    if not isinstance(v, dict):
        return v.float()
    codes = v["codes"].float()
    s = torch.exp2(v["scales"].float() - 127.0)
    return (codes.view(codes.shape[0], -1, 32) * s[:, :, None]).view_as(codes)


def _out_dtype(case):
    return torch.bfloat16 if case["dtype"] == "mx8" else _DTYPE[case["dtype"]]


def _written(v, case):
    """float32 rows as the case wants them: rounded once, or in 8 bits."""
    if case["out"] != "mx8":
        return v.to(_out_dtype(case))
    codes, scales = _quantise(v)
    return {"codes": codes, "scales": scales.view(torch.float8_e8m0fnu)}


def _sigmoid(v):
    return 1.0 / (1.0 + torch.exp(-v))


def _activate(v, act):
    if act == "silu":
        return v * _sigmoid(v)
    if act == "gelu":
        return 0.5 * v * (1.0 + torch.erf(v * 0.5 ** 0.5))
    if act == "relu2":
        return torch.clamp_min(v, 0.0) ** 2
    return v


def _slope(v, act):
    if act == "silu":
        s = _sigmoid(v)
        return s * (1.0 + v * (1.0 - s))
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(v * 0.5 ** 0.5)) + \
            v * torch.exp(-0.5 * v * v) * (2.0 * math.pi) ** -0.5
    return 2.0 * torch.clamp_min(v, 0.0)


def _halves(a, layout):
    if layout == "packed":
        return a.chunk(2, dim=1)
    return a[:, 0::2], a[:, 1::2]


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "norm":
        x, w = st["x"], st["weight"].float()
        if case["residual"]:
            x = (x.float() + st["residual"].float()).to(x.dtype)
        v = x.float()
        y = v * torch.rsqrt((v * v).mean(dim=1, keepdim=True) + _EPS) * w
        out = {"y": _written(y, case)}
        if case["residual"]:
            out["sum"] = x
        return out
    if op == "norm_grad":
        v, w, d = st["x"].float(), st["weight"].float(), st["d_y"].float()
        r = torch.rsqrt((v * v).mean(dim=1, keepdim=True) + _EPS)
        v = v * r
        dw = d * w
        d_x = r * (dw - v * (dw * v).mean(dim=1, keepdim=True))
        if case["residual"]:
            d_x = d_x + st["d_sum"].float()
        return {"d_x": d_x.to(st["x"].dtype), "d_weight": (d * v).sum(dim=0).to(st["x"].dtype)}
    if op in ("linear", "linear_grad"):
        x, w = _f32(st["x"]), _f32(st["w"])
        a = None
        if op == "linear" or case["act"] != "none":
            a = x @ w.t()
            if case["bias"]:
                a = a + st["bias"].float()
        if op == "linear":
            y = _activate(a, case["act"])
            if case["residual"]:
                y = y + st["residual"].float()
            return y.to(_out_dtype(case))
        d = st["d_y"].float()
        if a is not None:
            d = d * _slope(a, case["act"])
        t = st["x"].dtype
        out = {"d_x": (d @ w).to(t), "d_w": (d.t() @ x).to(t)}
        if case["bias"]:
            out["d_bias"] = d.sum(dim=0).to(t)
        return out
    x, w = _f32(st["x"]), _f32(st["w13"])
    g, u = _halves(x @ w.t(), case["layout"])
    oai = case["act"] == "swiglu_oai"
    if oai:
        gc, uc = torch.clamp_max(g, _LIMIT), torch.clamp(u, -_LIMIT, _LIMIT)
        s = _sigmoid(_ALPHA * gc)
    else:
        gc, uc, s = g, u, _sigmoid(g)
    up = uc + _BETA if oai else uc
    if op == "gated":
        return _written(gc * s * up, case)
    d = st["d_h"].float()
    d_g = d * up * s * (1.0 + (_ALPHA if oai else 1.0) * gc * (1.0 - s))
    d_u = d * gc * s
    if oai:
        d_g = torch.where(g <= _LIMIT, d_g, torch.zeros_like(d_g))
        d_u = torch.where(u.abs() <= _LIMIT, d_u, torch.zeros_like(d_u))
    if case["layout"] == "packed":
        d_a = torch.cat((d_g, d_u), dim=1)
    else:
        d_a = torch.stack((d_g, d_u), dim=2).flatten(1)
    t = st["x"].dtype
    return {"d_x": (d_a @ w).to(t), "d_w13": (d_a.t() @ x).to(t)}


# -------------------------------------------------------- the user's calls --

def _handles(st):
    """The row handles and the parameters that a user's program keeps."""
    if "handles" not in st:
        import mixture_experts_routing_warp_gb300 as moe

        case, h = st["case"], {}
        for name in ("x", "w", "w13"):
            if isinstance(st.get(name), dict):
                h[name] = moe.Mx8(st[name]["codes"], st[name]["scales"])
        if case["op"].startswith("gated"):
            h["params"] = moe.make_params(act=case["act"], layout=case["layout"])
        st["handles"] = h
    return st["handles"]


def _calls(st):
    import mixture_experts_routing_warp_gb300 as moe

    case, kept = st["case"], _handles(st)
    op = case["op"]

    def rows(name):
        return kept[name] if name in kept else st[name]

    def plain(y):
        if isinstance(y, moe.Mx8):
            return {"codes": y.codes, "scales": y.scales.view(torch.float8_e8m0fnu)}
        return y

    if op == "norm":
        got = moe.rms_norm(st["x"], st["weight"], _EPS, residual=st.get("residual"),
                           mx8=case["out"] == "mx8")
        if case["residual"]:
            return {"y": plain(got[0]), "sum": got[1]}
        return {"y": plain(got)}
    if op == "norm_grad":
        d_x, d_weight = moe.rms_norm_backward(st["d_y"], st["x"], st["weight"], _EPS,
                                              d_sum=st.get("d_sum"))
        return {"d_x": d_x, "d_weight": d_weight}
    if op == "linear":
        return moe.linear(rows("x"), rows("w"), bias=st.get("bias"), act=case["act"],
                          residual=st.get("residual"))
    if op == "linear_grad":
        d_x, d_w, d_bias = moe.linear_backward(st["d_y"], st["x"], st["w"], bias=st.get("bias"),
                                               act=case["act"])
        out = {"d_x": d_x, "d_w": d_w}
        if case["bias"]:
            out["d_bias"] = d_bias
        return out
    if op == "gated":
        return plain(moe.gated_linear(rows("x"), rows("w13"), kept["params"],
                                      mx8=case["out"] == "mx8"))
    d_x, d_w13 = moe.gated_linear_backward(st["d_h"], st["x"], st["w13"], kept["params"])
    return {"d_x": d_x, "d_w13": d_w13}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------- definition, 64 bit --

def _f64(v):
    if not isinstance(v, dict):
        return v.double()
    scale = torch.pow(2.0, v["scales"].double() - 127.0)
    return v["codes"].float().double() * torch.repeat_interleave(scale, 32, dim=1)


def _unrounded(v, case):
    """A row output before its last rounding. In 8 bits: the codes' values
    before they are rounded; a scale is either of two where a group's largest
    value lies at the border between them, so it has no such value."""
    if case["out"] != "mx8":
        return v
    top = v.unflatten(1, (-1, 32)).abs().amax(dim=2)
    e = torch.ceil(torch.log2(top / 448.0)).clamp_min(-127.0)
    return {"codes": v * torch.repeat_interleave(torch.pow(2.0, -e), 32, dim=1), "scales": None}


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op in ("norm", "norm_grad"):
        x, w = st["x"].double(), st["weight"].double()
        if op == "norm":
            total = x
            if case["residual"]:
                total = x + st["residual"].double()
                x = total.float().to(st["x"].dtype).double()   # the norm is of the rounded sum
            y = x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + _EPS) * w
            out = {"y": _unrounded(y, case)}
            if case["residual"]:
                out["sum"] = total
            return out
        x.requires_grad_()
        w.requires_grad_()
        with torch.enable_grad():
            y = x / torch.sqrt(x.square().mean(dim=1, keepdim=True) + _EPS) * w
            d_x, d_w = torch.autograd.grad(y, (x, w), st["d_y"].double())
        if case["residual"]:
            d_x = d_x + st["d_sum"].double()
        return {"d_x": d_x, "d_weight": d_w}
    x = _f64(st["x"]).requires_grad_()
    w = _f64(st["w" if op.startswith("linear") else "w13"]).requires_grad_()
    with torch.set_grad_enabled(op.endswith("grad")):
        a = torch.nn.functional.linear(x, w)
        if op.startswith("linear"):
            bias = st["bias"].double().requires_grad_() if case["bias"] else None
            if bias is not None:
                a = a + bias
            y = {"none": lambda v: v, "silu": torch.nn.functional.silu,
                 "gelu": torch.nn.functional.gelu,
                 "relu2": lambda v: torch.relu(v).square()}[case["act"]](a)
            if op == "linear":
                return y + st["residual"].double() if case["residual"] else y
            leaves = [x, w] + ([bias] if bias is not None else [])
            grads = torch.autograd.grad(y, leaves, st["d_y"].double())
            return dict(zip(("d_x", "d_w", "d_bias"), grads))
        I = case["I"]
        gate, up = (a[:, :I], a[:, I:]) if case["layout"] == "packed" else (a[:, ::2], a[:, 1::2])
        if case["act"] == "swiglu_oai":
            gate, up = gate.clamp(max=_LIMIT), up.clamp(-_LIMIT, _LIMIT)
            h = gate * torch.sigmoid(_ALPHA * gate) * (up + _BETA)
        else:
            h = torch.nn.functional.silu(gate) * up
        if op == "gated":
            return _unrounded(h, case)
        d_x, d_w = torch.autograd.grad(h, (x, w), st["d_h"].double())
    return {"d_x": d_x, "d_w13": d_w}
