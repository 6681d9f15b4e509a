"""The operators around the expert layer, as cases to time and to compare.

Three groups, each with its plain form in elementary torch operations and the
calls a user makes of `mixture_experts_routing_warp_gb300`:

  sorted tokens   dispatch (token rows -> expert-sorted rows) and combine_weighted
                  (sorted rows -> token rows, gate weights applied), with the
                  gradients of both
  route_backward  the gradient of the gate weights back to the router's logits
  4-bit weights   linear_q4 (a matrix-vector product for one or a few tokens) and
                  grouped_ffn_q4 (the experts of a decode step), E2M1 codes with
                  one E8M0 scale per 32 ("mxfp4") or one E4M3 scale per 16 and a
                  float per matrix ("nvfp4")
"""
import math

import torch

own = False

_BYTES = {"bf16": 2, "fp16": 2, "fp32": 4}
_DTYPE = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
_GROUP = {"mxfp4": 32, "nvfp4": 16}


# ------------------------------------------------------------------- cases --

def listed():
    return [
        # one decode step of 8 sequences, GPT-OSS layer: the rows fit any cache,
        # what counts is the call's latency
        dict(name="dispatch_n8_h2880", op="dispatch", n=8, H=2880, E=32, k=4, dtype="bf16",
             local=32),
        # the same layer's prefill: the row copy that feeds the experts' products
        dict(name="dispatch_n8192_h2880", op="dispatch", n=8192, H=2880, E=32, k=4, dtype="bf16",
             local=32),
        # gradient of the dispatch on an expert-parallel rank that holds 3 of 8
        # experts (float rows of a MiniMind layer in training, most slots elsewhere)
        dict(name="dispatch_grad_n4096_h512_fp32", op="dispatch_grad", n=4096, H=512, E=8, k=2,
             dtype="fp32", local=3),
        # 128 experts, skewed load: the largest prefill, back to token order
        dict(name="combine_n16384_h2880", op="combine", n=16384, H=2880, E=128, k=4, dtype="bf16",
             weights="bf16", local=128),
        # odd row length and slot count, half of the experts on another rank
        dict(name="combine_n517_h1001_fp16", op="combine", n=517, H=1001, E=16, k=3, dtype="fp16",
             weights="fp32", local=8),
        # training step of the GPT-OSS layer: both gradients of the weighted sum
        dict(name="combine_grad_n8192_h2880", op="combine_grad", n=8192, H=2880, E=32, k=4,
             dtype="bf16", weights="bf16", local=32),
        # the router's gradient at the layer sizes of the routing sweep
        dict(name="route_grad_n16384_e128_all", op="route_grad", n=16384, E=128, k=4,
             gating="softmax_all"),
        dict(name="route_grad_n33_e32_topk", op="route_grad", n=33, E=32, k=4,
             gating="softmax_topk"),
        # a projection beside the experts for one new token (latency), and for a
        # few with an odd number of rows
        dict(name="linear_q4_n1_2880x2880", op="linear_q4", n=1, R=2880, C=2880, fmt="mxfp4",
             dtype="bf16"),
        dict(name="linear_q4_n5_5761x1408", op="linear_q4", n=5, R=5761, C=1408, fmt="nvfp4",
             dtype="fp16"),
        # the GPT-OSS experts for one token, and for a decode batch of 64
        dict(name="ffn_q4_n1", op="ffn_q4", n=1, H=2880, I=2880, E=32, k=4, fmt="mxfp4",
             dtype="bf16", act="swiglu_oai", layout="interleaved", local=32),
        dict(name="ffn_q4_n64", op="ffn_q4", n=64, H=2880, I=2880, E=32, k=4, fmt="nvfp4",
             dtype="bf16", act="swiglu_oai", layout="interleaved", local=32),
    ]


def _log_int(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    done = [work(c) for c in listed()]
    top = {k: max(w[k] for w in done) for k in ("bytes", "flops")}
    while True:
        op = rng.choice(["dispatch", "dispatch_grad", "combine", "combine", "combine_grad",
                         "combine_grad", "route_grad", "linear_q4", "linear_q4", "ffn_q4",
                         "ffn_q4"])
        if op in ("dispatch", "dispatch_grad", "combine", "combine_grad"):
            E = _log_int(rng, 1, 256)
            k = min(E, rng.randint(1, 8))
            H = _log_int(rng, 1, 360) * 8 if rng.random() < 0.6 else _log_int(rng, 1, 2880)
            case = dict(op=op, n=_log_int(rng, 1, 16384), H=H, E=E, k=k,
                        dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                        local=E if rng.random() < 0.6 else rng.randint(1, E))
            if op.startswith("combine"):
                case["weights"] = rng.choice(["bf16", "fp32"])
        elif op == "route_grad":
            E = _log_int(rng, 1, 256)
            case = dict(op=op, n=_log_int(rng, 1, 16384), E=E, k=min(E, rng.randint(1, 8)),
                        gating=rng.choice(["softmax_topk", "softmax_all"]))
        elif op == "linear_q4":
            case = dict(op=op, n=_log_int(rng, 1, 24), R=_log_int(rng, 1, 16384),
                        C=32 * _log_int(rng, 1, 180), fmt=rng.choice(["mxfp4", "nvfp4"]),
                        dtype=rng.choice(["bf16", "fp16"]))
        else:
            E = _log_int(rng, 1, 64)
            case = dict(op=op, n=_log_int(rng, 1, 64), H=64 * _log_int(rng, 1, 45),
                        I=64 * _log_int(rng, 1, 45), E=E, k=min(E, rng.randint(1, 8)),
                        fmt=rng.choice(["mxfp4", "nvfp4"]), dtype=rng.choice(["bf16", "fp16"]),
                        act=rng.choice(["swiglu", "swiglu_oai", "relu2"]),
                        layout=rng.choice(["packed", "interleaved"]),
                        local=E if rng.random() < 0.7 else rng.randint(1, E))
        w = work(case)
        if w["bytes"] <= top["bytes"] and w["flops"] <= top["flops"]:
            if op != "ffn_q4" or case["local"] <= 32:
                return case


def work(case):
    op = case["op"]
    if op == "route_grad":
        n, E, k = case["n"], case["E"], case["k"]
        read = n * E * 4 if case["gating"] == "softmax_all" else n * k * 4
        return {"bytes": read + n * k * 8 + n * E * 4, "flops": 6 * n * (E + k)}
    if op == "linear_q4":
        n, R, C, s = case["n"], case["R"], case["C"], _BYTES[case["dtype"]]
        return {"bytes": R * C // 2 + R * C // _GROUP[case["fmt"]] + n * (R + C) * s,
                "flops": 2 * n * R * C}
    if op == "ffn_q4":
        n, H, I, E, k = (case[x] for x in ("n", "H", "I", "E", "k"))
        s, rows = _BYTES[case["dtype"]], I if case["act"] == "relu2" else 2 * I
        # experts with at least one slot, the slots drawn evenly
        hit = case["local"] * (1.0 - (1.0 - k / E) ** n)
        slots = n * k * case["local"] / E
        weights = (rows + I) * H
        return {"bytes": int(hit * (weights / 2 + weights / _GROUP[case["fmt"]]) + n * H * s +
                             n * k * (H * s + 8)),
                "flops": int(2 * slots * weights)}
    n, H, E, k, s = case["n"], case["H"], case["E"], case["k"], _BYTES[case["dtype"]]
    N, kept = n * k, n * k * case["local"] // E
    wb = N * _BYTES[case["weights"]] if "weights" in case else 0
    if op == "dispatch":  # rows of dropped slots at the end are zeros
        return {"bytes": n * H * s + N * H * s + N * 4, "flops": 0}
    if op == "dispatch_grad":
        return {"bytes": kept * H * s + n * H * s + N * 4, "flops": kept * H}
    if op == "combine":
        return {"bytes": kept * H * s + n * H * s + N * 4 + wb, "flops": 2 * kept * H}
    # combine_grad: out's gradient and the rows in, both gradients out
    return {"bytes": n * H * s + kept * H * s + N * H * s + N * 4 + wb + N * 4,
            "flops": 3 * kept * H}


# ------------------------------------------------------------------ inputs --

def _gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(0x5EED0000 + seed)
    return g


def _routing(case, g):
    """A routing as the layer builds it: top-k of random logits (skewed where
    there are 128 experts or more), and the metadata over the `local` experts
    that this rank holds; the slots of the others are dropped (-1)."""
    n, E, k, local = case["n"], case["E"], case["k"], case["local"]
    dev = "cuda"
    logits = torch.randn(n, E, generator=g, device=dev)
    if E >= 128:
        logits += 2.0 * torch.log(1.0 / (torch.arange(E, device=dev) + 1.0) ** 1.1)
    order = torch.argsort(logits, dim=1, descending=True, stable=True)
    indx = order[:, :k].to(torch.int32).contiguous()
    perm = torch.randperm(E, generator=g, device=dev)
    perm = torch.cat((indx[0, :1].long(), perm[perm != indx[0, 0]]))  # one slot at least is kept
    emap = torch.full((E,), -1, dtype=torch.int64, device=dev)
    emap[perm[:local]] = torch.arange(local, device=dev)
    if local == E:
        emap = torch.arange(E, device=dev)
    loc = emap[indx.long().reshape(-1)]                   # local expert of each slot, or -1
    kept = loc >= 0
    key = torch.where(kept, loc, torch.full_like(loc, local))
    col = torch.argsort(key, stable=True)                 # kept slots first, expert by expert
    row = torch.empty_like(col)
    row[col] = torch.arange(n * k, device=dev)
    row = torch.where(kept, row, torch.full_like(row, -1))
    count = torch.bincount(key, minlength=local + 1)[:local]
    offs = torch.zeros(local + 1, dtype=torch.int64, device=dev)
    offs[1:] = torch.cumsum(count, 0)
    col = torch.where(torch.arange(n * k, device=dev) < offs[-1], col, torch.zeros_like(col))
    sel = torch.gather(logits, 1, indx.long())
    vals = torch.softmax(sel, dim=1)
    meta = {"col_sum": count.to(torch.int32), "offs": offs.to(torch.int32),
            "col_sorted": col.to(torch.int32), "row_sorted": row.to(torch.int32),
            "gate_scal": vals.reshape(-1)[col].to(torch.bfloat16)}
    return logits, indx, vals, loc.reshape(n, k).to(torch.int32), meta


def _quantise(w, fmt):
    """Nearest E2M1 codes of w [R, C] under the format's group scales, as a
    checkpoint holds them: codes two per byte (even column low), scale bytes."""
    R, C = w.shape
    G = _GROUP[fmt]
    v = w.view(R, C // G, G)
    amax = v.abs().amax(dim=2).clamp_min(1e-12)
    if fmt == "mxfp4":
        e = torch.floor(torch.log2(amax)) - 2.0
        scales = (e + 127.0).to(torch.uint8)
        step = torch.exp2(e)
        whole = None
    else:
        whole = (amax.max() / (448.0 * 6.0)).reshape(1)
        q = (amax / 6.0 / whole).to(torch.float8_e4m3fn)
        scales = q.view(torch.uint8)
        step = q.float().clamp_min(2.0 ** -9) * whole
    u = v / step[:, :, None]
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device=w.device)
    code = torch.bucketize(u.abs(), mids) + 8 * (u < 0)
    code = code.view(R, C // 2, 2)
    return (code[:, :, 0] + 16 * code[:, :, 1]).to(torch.uint8), scales.contiguous(), whole


def _q4_matrices(count, R, C, fmt, g):
    codes = torch.empty(count, R, C // 2, dtype=torch.uint8, device="cuda")
    scales = torch.empty(count, R, C // _GROUP[fmt], dtype=torch.uint8, device="cuda")
    whole = torch.ones(count, dtype=torch.float32, device="cuda")
    for e in range(count):
        w = torch.randn(R, C, generator=g, device="cuda") * 0.02
        codes[e], scales[e], s = _quantise(w, fmt)
        if s is not None:
            whole[e:e + 1] = s
    return {"codes": codes, "scales": scales, "matrix_scale": whole if fmt == "nvfp4" else None}


def prepare(case, seed):
    g = _gen(seed)
    op = case["op"]
    st = {"case": case}
    if op == "linear_q4":
        st["x"] = torch.randn(case["n"], case["C"], generator=g, device="cuda").to(
            _DTYPE[case["dtype"]])
        w = _q4_matrices(1, case["R"], case["C"], case["fmt"], g)
        st["w"] = {k: (v[0] if v is not None and v.dim() > 1 else v) for k, v in w.items()}
    elif op == "route_grad":
        full = dict(case, local=case["E"])
        logits, indx, vals, _, _ = _routing(full, g)
        st.update(logits=logits, indx=indx,
                  d_vals=torch.randn(case["n"], case["k"], generator=g, device="cuda"))
    else:
        dt = _DTYPE[case["dtype"]]
        n, H, k = case["n"], case["H"], case["k"]
        _, _, vals, loc, meta = _routing(case, g)
        st.update(meta=meta, loc=loc)
        if op == "ffn_q4":
            rows = case["I"] if case["act"] == "relu2" else 2 * case["I"]
            st["x"] = torch.randn(n, H, generator=g, device="cuda").to(dt)
            st["w13"] = _q4_matrices(case["local"], rows, H, case["fmt"], g)
            st["w2"] = _q4_matrices(case["local"], H, case["I"], case["fmt"], g)
        elif op == "dispatch":
            st["x"] = torch.randn(n, H, generator=g, device="cuda").to(dt)
        else:
            st["rows"] = torch.randn(n * k, H, generator=g, device="cuda").to(dt)
            if op.startswith("combine"):
                st["weights"] = vals.to(_DTYPE[case["weights"]])
            if op == "combine_grad":
                st["d_out"] = torch.randn(n, H, generator=g, device="cuda").to(dt)
    if own:
        _handles(st)
    return st


def _handles(st):
    """The weight handles and the workspace that a serving program keeps."""
    if "handles" in st:
        return st["handles"]
    import mixture_experts_routing_warp_gb300 as moe

    case, h = st["case"], {}
    for name in ("w", "w13", "w2"):
        if name in st:
            h[name] = moe.Q4Weight(st[name]["codes"], st[name]["scales"], case["fmt"],
                                   st[name]["matrix_scale"])
    if case["op"] == "ffn_q4":
        h["params"] = moe.make_params("softmax_topk", case["act"], case["layout"])
        h["ws"] = moe.workspace_q4(case["n"], case["local"], case["k"], case["H"], case["I"])
    st["handles"] = h
    return h


# ------------------------------------------------------------- plain forms --

def _decode_q4(codes, scales, fmt, whole):
    """float32 [R, C] of one matrix."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0,
                          -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=codes.device)
    R, half = codes.shape
    lo, hi = (codes & 15).int(), (codes >> 4).int()
    v = torch.stack((table[lo], table[hi]), dim=2).view(R, -1, _GROUP[fmt])
    if fmt == "mxfp4":
        s = torch.exp2(scales.float() - 127.0)
    else:
        s = scales.view(torch.float8_e4m3fn).float() * whole
    return (v * s[:, :, None]).view(R, 2 * half)


def _activate(a, act, layout):
    if act == "relu2":
        return torch.clamp_min(a, 0.0) ** 2
    if layout == "packed":
        g, u = a.chunk(2, dim=1)
    else:
        g, u = a[:, 0::2], a[:, 1::2]
    if act == "swiglu_oai":
        g, u = torch.clamp_max(g, 7.0), torch.clamp(u, -7.0, 7.0)
        return g / (1.0 + torch.exp(-1.702 * g)) * (u + 1.0)
    return g / (1.0 + torch.exp(-g)) * u


def _plain(st):
    case = st["case"]
    op = case["op"]
    if op == "linear_q4":
        w = _decode_q4(st["w"]["codes"], st["w"]["scales"], case["fmt"], st["w"]["matrix_scale"])
        return (st["x"].float() @ w.t()).to(st["x"].dtype)
    if op == "route_grad":
        logits, idx, d = st["logits"], st["indx"].long(), st["d_vals"]
        sel = torch.gather(logits, 1, idx)
        src = sel if case["gating"] == "softmax_topk" else logits
        top = src.amax(dim=1, keepdim=True)
        den = torch.exp(src - top).sum(dim=1, keepdim=True)
        p = torch.exp(sel - top) / den
        mean = (p * d).sum(dim=1, keepdim=True)
        if case["gating"] == "softmax_topk":
            return torch.zeros_like(logits).scatter_(1, idx, p * (d - mean))
        out = -mean * (torch.exp(logits - top) / den)
        return out.scatter_add_(1, idx, p * d)
    meta, n, H, k = st["meta"], case["n"], case["H"], case["k"]
    row = meta["row_sorted"].long()
    live = (row >= 0)[:, None]
    at = row.clamp_min(0)
    col = meta["col_sorted"].long()
    kept = (torch.arange(n * k, device=col.device) < meta["offs"][-1])[:, None]
    if op == "ffn_q4":
        x, loc = st["x"].float(), st["loc"]
        y = torch.zeros(n, k, H, device="cuda")
        w13, w2 = st["w13"], st["w2"]
        # the experts to visit: each slot's own when the slots are fewer
        slots = loc.reshape(-1).clamp_min(0).long()
        visit = slots if slots.numel() < case["local"] else torch.arange(case["local"],
                                                                         device="cuda")
        for i in range(visit.numel()):
            e = visit[i:i + 1]

            def matrix(w):
                whole = w["matrix_scale"]
                return _decode_q4(w["codes"].index_select(0, e)[0],
                                  w["scales"].index_select(0, e)[0], case["fmt"],
                                  whole if whole is None else whole.index_select(0, e))

            a = x @ matrix(w13).t()
            h = _activate(a, case["act"], case["layout"])
            o = h @ matrix(w2).t()
            y = torch.where((loc == e)[:, :, None], o[:, None, :], y)
        y = torch.where(kept, y.view(n * k, H)[col], torch.zeros((), device="cuda"))
        return y.to(st["x"].dtype)
    if op == "dispatch":
        x = st["x"]
        return torch.where(kept, x[torch.div(col, k, rounding_mode="floor")], torch.zeros_like(x[:1]))
    if op in ("dispatch_grad", "combine"):
        rows = torch.where(live, st["rows"][at].float(), torch.zeros((), device="cuda"))
        if op == "combine":
            rows = rows * st["weights"].float().reshape(-1, 1)
        return rows.view(n, k, H).sum(dim=1).to(st["rows"].dtype)
    d_out, w = st["d_out"].float(), st["weights"].float().reshape(-1, 1)
    up = d_out[:, None, :].expand(n, k, H).reshape(n * k, H)
    d_flat = w * up
    d_rows = torch.where(kept, d_flat[col], torch.zeros((), device="cuda")).to(st["rows"].dtype)
    rows = torch.where(live, st["rows"][at].float(), torch.zeros((), device="cuda"))
    return {"d_sorted": d_rows, "d_weights": (rows * up).sum(dim=1).view(n, k)}


# -------------------------------------------------------- the user's calls --

def _calls(st):
    import mixture_experts_routing_warp_gb300 as moe

    case, h = st["case"], _handles(st)
    op = case["op"]
    if op == "linear_q4":
        return moe.linear_q4(st["x"], h["w"])
    if op == "route_grad":
        return moe.route_backward(st["logits"], st["indx"], st["d_vals"], case["gating"])
    if op == "ffn_q4":
        return moe.grouped_ffn_q4(st["x"], st["meta"], h["w13"], h["w2"], case["k"], h["ws"],
                                  h["params"])
    if op == "dispatch":
        return moe.dispatch(st["x"], st["meta"], case["k"])
    if op == "dispatch_grad":
        return moe.dispatch_backward(st["rows"], st["meta"], case["k"])
    if op == "combine":
        return moe.combine_weighted(st["rows"], st["meta"], st["weights"])
    d_sorted, d_weights = moe.combine_weighted_backward(st["d_out"], st["rows"], st["meta"],
                                                        st["weights"])
    return {"d_sorted": d_sorted, "d_weights": d_weights}


def run(state):
    return _calls(state) if own else _plain(state)


# ------------------------------------------------------- definition, 64 bit --

def _value64(codes, scales, fmt, whole):
    """A code's value from its bits: sign, two exponent bits, one mantissa bit."""
    nib = torch.stack((codes % 16, codes // 16), dim=-1).flatten(1).double()
    neg = nib >= 8
    mag = nib - 8.0 * neg
    e = torch.floor(mag / 2)
    m = mag - 2 * e
    v = torch.where(e == 0, 0.5 * m, torch.pow(2.0, e - 1) * (1 + 0.5 * m))
    v = torch.where(neg, -v, v)
    if fmt == "mxfp4":
        s = torch.pow(2.0, scales.double() - 127.0)
    else:
        b = scales.double()
        sneg = b >= 128
        b = b - 128 * sneg
        se = torch.floor(b / 8)
        sm = b - 8 * se
        s = torch.where(se == 0, sm * 2.0 ** -9, torch.pow(2.0, se - 7) * (1 + sm / 8))
        s = torch.where(sneg, -s, s) * whole.double()
    return v * torch.repeat_interleave(s, _GROUP[fmt], dim=1)


def exact(case, seed):
    st = prepare(case, seed)
    op = case["op"]
    if op == "linear_q4":
        w = st["w"]
        return st["x"].double() @ _value64(w["codes"], w["scales"], case["fmt"],
                                           w["matrix_scale"]).t()
    if op == "route_grad":
        z, idx, d = st["logits"].double(), st["indx"].long(), st["d_vals"].double()
        chosen = torch.zeros_like(z, dtype=torch.bool).scatter_(1, idx, True)
        up = torch.zeros_like(z).scatter_(1, idx, d)
        if case["gating"] == "softmax_topk":
            z = z.masked_fill(~chosen, -math.inf)
        p = torch.softmax(z, dim=1)
        return p * (up - (p * up).sum(dim=1, keepdim=True))
    meta, n, H, k = st["meta"], case["n"], case["H"], case["k"]
    offs = meta["offs"].tolist()
    total = offs[-1]
    slot = meta["col_sorted"][:total].long()
    token = torch.div(slot, k, rounding_mode="floor")
    if op == "ffn_q4":
        out = torch.zeros(n * k, H, dtype=torch.float64, device="cuda")
        for e in range(case["local"]):
            lo, hi = offs[e], offs[e + 1]
            if lo == hi:
                continue
            m = [None, None] if case["fmt"] == "mxfp4" else [st[w]["matrix_scale"][e]
                                                             for w in ("w13", "w2")]
            a = st["x"][token[lo:hi]].double() @ _value64(
                st["w13"]["codes"][e], st["w13"]["scales"][e], case["fmt"], m[0]).t()
            if case["act"] == "relu2":
                h = torch.relu(a).square()
            else:
                I = case["I"]
                g, u = (a[:, :I], a[:, I:]) if case["layout"] == "packed" else (a[:, ::2],
                                                                              a[:, 1::2])
                if case["act"] == "swiglu_oai":
                    g = torch.minimum(g, torch.full_like(g, 7.0))
                    u = u.clamp(-7.0, 7.0)
                    h = g * torch.sigmoid(1.702 * g) * (u + 1.0)
                else:
                    h = g * torch.sigmoid(g) * u
            out[lo:hi] = h @ _value64(st["w2"]["codes"][e], st["w2"]["scales"][e], case["fmt"],
                                      m[1]).t()
        return out
    if op == "dispatch":
        out = torch.zeros(n * k, H, dtype=torch.float64, device="cuda")
        out[:total] = st["x"].double()[token]
        return out
    if op in ("dispatch_grad", "combine"):
        src = st["rows"][:total].double()
        if op == "combine":
            src = src * st["weights"].double().reshape(-1)[slot][:, None]
        return torch.zeros(n, H, dtype=torch.float64, device="cuda").index_add_(0, token, src)
    d_out = st["d_out"].double()
    d_sorted = torch.zeros(n * k, H, dtype=torch.float64, device="cuda")
    d_sorted[:total] = d_out[token] * st["weights"].double().reshape(-1)[slot][:, None]
    d_w = torch.zeros(n * k, dtype=torch.float64, device="cuda")
    d_w[slot] = (d_out[token] * st["rows"][:total].double()).sum(dim=1)
    return {"d_sorted": d_sorted, "d_weights": d_w.view(n, k)}
