"""Products with 4-bit weights (moe.linear_q4, moe.grouped_ffn_q4,
moe.forward_q4) against the definition in 64 bits.

Tolerances. The weights are exact. An activation row is scaled to a largest
magnitude of at least 2^14 and stored as fp16: bf16 and fp16 values change by
at most half of fp16's smallest step, 2^-25, that is 2^-39 of the row's
maximum; fp32 values (h) also by fp16's half step, 2^-11 of themselves. Each
16-product instruction and each join of partial sums rounds or truncates one
fp32 sum, 2^-23 of the magnitudes summed; a result is rounded once to its
type, eps / 2."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe

pytestmark = pytest.mark.gpu

GROUP = {"mxfp4": 32, "nvfp4": 16}
BF16, FP16 = torch.bfloat16, torch.float16
VALUES = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def random_q4(shape, fmt, seed, spread=4, count=None):
    """Codes of every value, scales over 2^spread binary orders."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    lead, (R, C) = (() if count is None else (count,)), shape
    codes = torch.randint(0, 256, (*lead, R, C // 2), generator=g, device="cuda",
                          dtype=torch.uint8)
    if fmt == "mxfp4":
        scales = torch.randint(120 - spread, 121, (*lead, R, C // 32), generator=g, device="cuda",
                               dtype=torch.uint8)
        whole = None
    else:   # E4M3 codes of both signs but NaN; a scale may be negative or zero
        scales = torch.randint(0, 127, (*lead, R, C // 16), generator=g, device="cuda",
                               dtype=torch.uint8)
        scales += 128 * torch.randint(0, 2, scales.shape, generator=g, device="cuda",
                                      dtype=torch.uint8)
        whole = torch.rand(count or 1, generator=g, device="cuda") * 1e-3 + 1e-4
    return moe.Q4Weight(codes, scales, fmt, whole)


def decode64(w, e=0):
    codes = w.codes if w.codes.dim() == 2 else w.codes[e]
    scales = w.scales if w.scales.dim() == 2 else w.scales[e]
    nib = torch.stack((codes & 15, codes >> 4), -1).flatten(1).long()
    v = torch.tensor(VALUES + [-x for x in VALUES], dtype=torch.float64, device="cuda")[nib]
    if w.fmt == "mxfp4":
        s = torch.where(scales == 255, torch.nan, torch.exp2(scales.double() - 127))
    else:
        s = scales.view(torch.float8_e4m3fn).double()
        if w.matrix_scale is not None:
            s = s * w.matrix_scale.double()[e]
    return v * s.repeat_interleave(GROUP[w.fmt], 1)


def product64(x, W, fp32_in=False):
    """x W^T and the bound on its error before the last rounding."""
    ref, mag = x @ W.t(), x.abs() @ W.abs().t()
    top = x.abs().amax(1, keepdim=True) if x.shape[0] else x[:, :1]
    C = x.shape[1]
    err = (C / 16 + 16) * 2.0 ** -23 * mag + 2.0 ** -39 * top * W.abs().sum(1)
    return ref, err + (2.0 ** -11 * mag if fp32_in else 0.0)


def check(got, ref, err):
    u, dt = torch.finfo(got.dtype).eps / 2, got.dtype
    tiny = 2.0 ** -25 if dt == FP16 else 2.0 ** -134
    diff = (got.double() - ref).abs()
    tol = err + u * (ref.abs() + err) + tiny
    assert (diff <= tol).all(), (diff / tol).max().item()


def tokens(n, C, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(n, C, generator=g, device="cuda") * scale).to(dtype)


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_every_weight_comes_through_exactly(fmt):
    """Unit vectors read the weights out one by one: bf16 holds an E2M1 value
    times a power of two, fp16 an E2M1 value times an E4M3 one."""
    for C in (32, 96, 128, 416):
        w = random_q4((75, C), fmt, C)
        w = moe.Q4Weight(w.codes, w.scales, fmt)
        x = torch.eye(C, device="cuda", dtype=BF16 if fmt == "mxfp4" else FP16)
        got = moe.linear_q4(x, w)
        assert torch.equal(got.double(), decode64(w).t())


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("n,R,C", [(1, 1, 32), (1, 2880, 2880), (2, 17, 64), (3, 15, 160),
                                   (7, 5761, 1408), (8, 333, 512), (9, 64, 288), (16, 129, 1024),
                                   (17, 257, 2880), (40, 31, 352), (1, 40000, 96), (5, 48, 5760)])
def test_linear(n, R, C, fmt, dtype):
    w, x = random_q4((R, C), fmt, 1), tokens(n, C, dtype, 2)
    check(moe.linear_q4(x, w), *product64(x.double(), decode64(w)))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("n", [1, 3, 20])
def test_rows_longer_than_the_resident_activations(fmt, n):
    w, x = random_q4((35, 20000), fmt, 3), tokens(n, 20000, BF16, 4)
    check(moe.linear_q4(x, w), *product64(x.double(), decode64(w)))


@pytest.mark.parametrize("n", [1, 12])
def test_scales_far_apart(n):
    """Group scales of one row up to 2^100 apart, with activations that make
    the small groups count: each slab's sum keeps its own scale."""
    C = 416
    w, x = random_q4((50, C), "mxfp4", 5), tokens(n, C, BF16, 6)
    g = torch.Generator(device="cuda")
    g.manual_seed(7)
    w.scales.copy_(torch.randint(77, 178, w.scales.shape, generator=g, device="cuda",
                                 dtype=torch.uint8))
    W = decode64(w)
    out = moe.linear_q4(x, w)
    check(out, *product64(x.double(), W))
    # only the row's smallest group is touched: nothing larger hides its error
    for r in (0, 31, 49):
        j = int(w.scales[r].argmin())
        cols = slice(32 * j, 32 * j + 32)
        only = torch.zeros_like(x)
        only[:, cols] = x[:, cols]
        ref, err = product64(x[:, cols].double(), W[r:r + 1, cols])
        check(moe.linear_q4(only, w)[:, r:r + 1], ref, err)


def test_extreme_scales_and_nan():
    """Scale bytes 0 (2^-127) and 223 (2^96, the largest supported), and NaN
    scales: a NaN reaches its own row and no other."""
    C = 160
    w = random_q4((40, C), "mxfp4", 8)
    w.scales[3] = 0
    w.scales[4, 1], w.scales[5, 4] = 255, 255
    x = tokens(2, C, BF16, 9, 2.0 ** 20)
    out, W = moe.linear_q4(x, w), decode64(w)
    assert out[:, 4:6].isnan().all()
    keep = [r for r in range(40) if r not in (4, 5)]
    check(out[:, keep], *product64(x.double(), W[keep]))
    w.scales[7] = 223
    x = tokens(2, C, BF16, 9, 2.0 ** -30)
    ref, err = product64(x.double(), decode64(w)[7:8])
    check(moe.linear_q4(x, w)[:, 7:8], ref, err)
    v = random_q4((40, C), "nvfp4", 10)
    v.scales[6, 9], v.scales[9, 0] = 127, 255
    out, W = moe.linear_q4(x, v), decode64(v)
    assert out[:, [6, 9]].isnan().all()
    keep = [r for r in range(40) if r not in (6, 9)]
    check(out[:, keep], *product64(x.double(), W[keep]))


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
def test_activation_rows_of_every_size(fmt):
    """Rows of zeros, of subnormals, near the type's largest value, and rows
    whose entries differ by many orders."""
    C = 256
    w = random_q4((64, C), fmt, 11)
    if fmt == "nvfp4":
        w = moe.Q4Weight(w.codes, w.scales, fmt, torch.full((1,), 2.0 ** -20, device="cuda"))
    else:
        w.scales.fill_(100)
    x = tokens(7, C, BF16, 12)
    x[0] = 0
    x[1] *= 2.0 ** -100
    x[2] *= 2.0 ** 100
    x[3] *= torch.exp2(-torch.arange(C, device="cuda") / 8.0).to(BF16)
    x[4, 1:] = 0
    x[5] = torch.finfo(BF16).max * 2.0 ** -12
    check(moe.linear_q4(x, w), *product64(x.double(), decode64(w)))


def test_infinities_and_nan_stay_in_their_token():
    C = 192
    for fmt in ("mxfp4", "nvfp4"):
        w, x = random_q4((33, C), fmt, 13), tokens(5, C, BF16, 14)
        w.codes[:, 20] = 0x11   # columns 40, 41: no zero weight under the infinity
        clean = moe.linear_q4(x, w)
        y = x.clone()
        y[1, 3], y[3, 40] = float("nan"), float("inf")
        out = moe.linear_q4(y, w)
        assert out[1].isnan().all()
        for t in (0, 2, 4):
            assert torch.equal(out[t], clean[t])
        col = decode64(w)[:, 40]
        nonzero = col != 0
        assert torch.equal(out[3][nonzero], (col[nonzero] * float("inf")).to(BF16))


# ------------------------------------------------------------- the experts --

def make_meta(n, E, k, seed, local=None, skew=False):
    rng = np.random.default_rng(seed)
    p = np.arange(1, E + 1) ** -1.5 if skew else np.ones(E)
    indx = np.stack([rng.choice(E, k, replace=False, p=p / p.sum()) for _ in range(n)])
    local = E if local is None else local
    flat = indx.reshape(-1)
    col = [f for e in range(local) for f in np.nonzero(flat == e)[0]]
    row = np.full(n * k, -1)
    row[col] = np.arange(len(col))
    offs = np.zeros(local + 1)
    offs[1:] = np.cumsum([(flat == e).sum() for e in range(local)])
    # the entries past the kept slots hold anything
    full = np.concatenate([col, rng.integers(-2 ** 31, 2 ** 31, n * k - len(col))])
    t = lambda a: torch.from_numpy(np.asarray(a).astype(np.int32)).cuda()
    return {"row_sorted": t(row), "offs": t(offs), "col_sorted": t(full)}


def activate64(a, err, act, layout, limit):
    """act(a) and the bound on its error: the inputs' error times the slope,
    and 2^-19 for the fp32 evaluation (an exponential and a reciprocal of a
    few ulp each, the argument's rounding times its size)."""
    if act == "relu2":
        h = a.clamp_min(0) ** 2
        return h, 2 * a.abs() * err + err ** 2 + 2.0 ** -22 * h
    I = a.shape[1] // 2
    pick = (lambda t: (t[:, :I], t[:, I:])) if layout == "packed" else \
        (lambda t: (t[:, 0::2], t[:, 1::2]))
    (g, up), (eg, eu) = pick(a), pick(err)
    alpha, beta = 1.0, 0.0
    if act == "swiglu_oai":
        alpha, beta, limit = 1.702, 1.0, 7.0
    if limit is not None:
        g, up = g.clamp_max(limit), up.clamp(-limit, limit)
    s = torch.sigmoid(alpha * g)
    h = g * s * (up + beta)
    return h, 1.2 * (up + beta).abs() * eg + (g * s).abs() * eu + eg * eu + 2.0 ** -19 * (
        h.abs() + (g * s).abs())


def ffn64(x, meta, w13, w2, k, act, layout, limit=None):
    offs, N = meta["offs"].tolist(), meta["row_sorted"].numel()
    H = x.shape[1]
    y = torch.zeros(N, H, dtype=torch.float64, device="cuda")
    tol = torch.zeros_like(y)
    for e in range(len(offs) - 1):
        lo, hi = offs[e], offs[e + 1]
        if lo == hi:
            continue
        tok = meta["col_sorted"][lo:hi].long() // k
        a, ea = product64(x[tok].double(), decode64(w13, e))
        h, eh = activate64(a, ea, act, layout, limit)
        W2 = decode64(w2, e)
        y[lo:hi], err = product64(h, W2, fp32_in=True)
        tol[lo:hi] = err + eh @ W2.abs().t()
    return y, tol


CASES = [  # n, H, I, E, k, local, skew
    (1, 64, 64, 4, 2, 4, False), (1, 2880, 2880, 8, 4, 8, False), (3, 192, 320, 5, 3, 5, False),
    (8, 512, 1408, 16, 2, 16, False), (33, 128, 64, 8, 4, 3, False),
    (64, 320, 192, 32, 4, 32, True), (200, 64, 128, 3, 1, 3, True),
    (70, 128, 192, 256, 8, 256, False), (19, 576, 64, 2, 2, 1, False)]


@pytest.mark.parametrize("act,layout,limit", [
    ("swiglu", "packed", None), ("swiglu", "interleaved", 2.0), ("swiglu_oai", "interleaved", None),
    ("swiglu_oai", "packed", None), ("relu2", "packed", None)])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("n,H,I,E,k,local,skew", CASES)
def test_grouped_ffn(n, H, I, E, k, local, skew, fmt, act, layout, limit):
    dtype = BF16 if (n + H) % 128 else FP16
    meta = make_meta(n, E, k, 20, local, skew)
    w13 = random_q4((I if act == "relu2" else 2 * I, H), fmt, 21, count=local)
    w2 = random_q4((H, I), fmt, 22, count=local)
    x = tokens(n, H, dtype, 23, 0.1)
    ws = moe.workspace_q4(n, local, k, H, I)
    p = moe.make_params(act=act, layout=layout, limit=limit)
    got = moe.grouped_ffn_q4(x, meta, w13, w2, k, ws, p)
    ref, tol = ffn64(x, meta, w13, w2, k, act, layout, limit)
    check(got, ref, tol)
    assert (got[int(meta["offs"][-1]):] == 0).all()


def test_formats_may_differ_between_the_two_products():
    n, H, I, E, k = 5, 128, 192, 4, 2
    meta, x = make_meta(n, E, k, 30), tokens(n, H, BF16, 31, 0.1)
    w13 = random_q4((2 * I, H), "nvfp4", 32, count=E)
    w2 = random_q4((H, I), "mxfp4", 33, count=E)
    got = moe.grouped_ffn_q4(x, meta, w13, w2, k, moe.workspace_q4(n, E, k, H, I),
                             moe.make_params())
    check(got, *ffn64(x, meta, w13, w2, k, "swiglu", "packed"))


def test_no_tokens_and_no_slots():
    w = random_q4((48, 64), "mxfp4", 40)
    assert moe.linear_q4(torch.empty(0, 64, dtype=BF16, device="cuda"), w).shape == (0, 48)
    E, k, H, I = 3, 2, 64, 64
    w13, w2 = random_q4((2 * I, H), "nvfp4", 41, count=E), random_q4((H, I), "nvfp4", 42, count=E)
    for n in (0, 4):   # no token; tokens whose slots are all dropped
        meta = {"offs": torch.zeros(E + 1, dtype=torch.int32, device="cuda"),
                "col_sorted": torch.full((n * k,), -7, dtype=torch.int32, device="cuda")}
        got = moe.grouped_ffn_q4(tokens(n, H, BF16, 43), meta, w13, w2, k,
                                 moe.workspace_q4(n, E, k, H, I), moe.make_params())
        assert got.shape == (n * k, H) and (got == 0).all()


def test_broken_metadata_stays_inside_the_buffers():
    """Offsets and slots out of range or out of order give unspecified rows,
    but no access outside the arrays (canaries around every output)."""
    n, H, I, E, k = 6, 64, 64, 4, 2
    w13, w2 = random_q4((2 * I, H), "mxfp4", 44, count=E), random_q4((H, I), "mxfp4", 45, count=E)
    x = tokens(n, H, BF16, 46)
    N, size = n * k, moe.workspace_q4_size(n, E, k, H, I)
    raw = torch.full((size + 8192,), 0xA5, dtype=torch.uint8, device="cuda")
    ws = raw[4096:4096 + size]
    assert moe.lib().moe_workspace_init(ws.data_ptr(), size, None) == 0
    out_raw = torch.full((N * H + 4096,), 7.0, dtype=BF16, device="cuda")
    out = out_raw[2048:2048 + N * H].view(N, H)
    for offs in ([0, 5, 3, 2 ** 31 - 1, 12], [-9, -9, 40, 1, -1], [12, 12, 0, 0, 12]):
        meta = {"offs": torch.tensor(offs, dtype=torch.int32).cuda(),
                "col_sorted": torch.tensor([2 ** 31 - 1, -(2 ** 31)] * (N // 2),
                                           dtype=torch.int32).cuda()}
        moe.grouped_ffn_q4(x, meta, w13, w2, k, ws, moe.make_params(), out=out)
        torch.cuda.synchronize()
        assert (raw[:4096] == 0xA5).all() and (raw[4096 + size:] == 0xA5).all()
        assert (out_raw[:2048] == 7).all() and (out_raw[2048 + N * H:] == 7).all()


@pytest.mark.parametrize("n", [1, 9])
def test_outputs_stay_inside_their_rows(n):
    """Odd row counts: nothing before or after the output is written."""
    R, C = 83, 160
    w, x = random_q4((R, C), "nvfp4", 47), tokens(n, C, FP16, 48)
    raw = torch.full((n * R + 4096,), 7.0, dtype=FP16, device="cuda")
    out = raw[2047:2047 + n * R].view(n, R)   # aligned to its element only
    moe.linear_q4(x, w, out=out)
    assert (raw[:2047] == 7).all() and (raw[2047 + n * R:] == 7).all()
    assert torch.equal(out, moe.linear_q4(x, w))


def test_offsets_past_32_bits():
    """More than 2^32 bytes of codes: the last experts' weights are the ones
    read."""
    E, H, I, n, k = 250, 4096, 4224, 4, 2
    codes = torch.zeros(E, 2 * I, H // 2, dtype=torch.uint8, device="cuda")
    assert codes.numel() > 2 ** 32
    w13 = random_q4((2 * I, H), "mxfp4", 50, count=1)
    scales = torch.full((E, 2 * I, H // 32), 118, dtype=torch.uint8, device="cuda")
    codes[E - 1], scales[E - 1] = w13.codes[0], w13.scales[0]
    c2 = torch.zeros(E, H, I // 2, dtype=torch.uint8, device="cuda")
    s2 = torch.full((E, H, I // 32), 118, dtype=torch.uint8, device="cuda")
    w2 = random_q4((H, I), "mxfp4", 51, count=1)
    c2[E - 1], s2[E - 1] = w2.codes[0], w2.scales[0]
    x = tokens(n, H, BF16, 52, 0.1)
    N = n * k
    offs = torch.zeros(E + 1, dtype=torch.int32, device="cuda")
    offs[E] = N
    offs[E - 1] = N - 3
    offs[1:E - 1] = N - 3
    meta = {"offs": offs, "row_sorted": torch.arange(N, dtype=torch.int32, device="cuda"),
            "col_sorted": torch.arange(N, dtype=torch.int32, device="cuda")}
    got = moe.grouped_ffn_q4(x, meta, moe.Q4Weight(codes, scales, "mxfp4"),
                             moe.Q4Weight(c2, s2, "mxfp4"), k,
                             moe.workspace_q4(n, E, k, H, I), moe.make_params())
    one = {"offs": torch.tensor([0, 3], dtype=torch.int32, device="cuda"),
           "row_sorted": torch.arange(3, dtype=torch.int32),
           "col_sorted": meta["col_sorted"][N - 3:]}
    ref, tol = ffn64(x, one, w13, w2, k, "swiglu", "packed")
    check(got[N - 3:], ref, tol)
    assert (got[:N - 3] == 0).all()   # expert 0's codes are zeros


def test_streams_graphs_and_repeats():
    n, H, I, E, k = 6, 320, 192, 8, 2
    w13, w2 = random_q4((2 * I, H), "nvfp4", 60, count=E), random_q4((H, I), "nvfp4", 61, count=E)
    p, ws = moe.make_params(), moe.workspace_q4(n, E, k, H, I)
    x, z = tokens(n, H, BF16, 62, 0.1), torch.randn(n, E, device="cuda")
    first = moe.forward_q4(x, z, w13, w2, k, p, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = moe.forward_q4(x, z, w13, w2, k, p, ws)
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(first, second)
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(first)
    with torch.cuda.graph(graph):
        moe.forward_q4(x, z, w13, w2, k, p, ws, out=out)
    x.copy_(tokens(n, H, BF16, 63, 0.1))
    z.copy_(torch.randn(n, E, device="cuda"))
    graph.replay()
    assert torch.equal(out, moe.forward_q4(x, z, w13, w2, k, p, ws))


def test_two_streams_at_a_time():
    """Layers on two streams, each with a workspace of its own, do not wait
    for one another's halves (a launch has all its blocks resident)."""
    n, H, I, E, k = 4, 256, 256, 8, 2
    w13, w2 = random_q4((2 * I, H), "mxfp4", 64, count=E), random_q4((H, I), "mxfp4", 65, count=E)
    p = moe.make_params()
    x, z = tokens(n, H, BF16, 66, 0.1), torch.randn(n, E, device="cuda")
    spaces = [moe.workspace_q4(n, E, k, H, I) for _ in range(2)]
    want = moe.forward_q4(x, z, w13, w2, k, p, spaces[0])
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(2)], []
    for i in range(40):
        with torch.cuda.stream(streams[i % 2]):
            outs.append(moe.forward_q4(x, z, w13, w2, k, p, spaces[i % 2]))
    torch.cuda.synchronize()
    for ws in spaces:
        assert moe.read_status(ws) == 0
    for out in outs:
        assert torch.equal(out, want)


@pytest.mark.parametrize("n,local", [(1, 16), (7, 16), (64, 16), (40, 5)])
@pytest.mark.parametrize("gating", ["softmax_topk", "softmax_all"])
def test_forward_is_its_stages(n, local, gating):
    """moe.forward_q4 = routing, grouped_ffn_q4, combine_weighted, with the
    routing's outputs handed out; and the layer in 64 bits."""
    H, I, E, k = 256, 192, 16, 4
    w13 = random_q4((2 * I, H), "mxfp4", 70, count=local)
    w2 = random_q4((H, I), "mxfp4", 71, count=local)
    x = tokens(n, H, BF16, 72, 0.1)
    z = torch.randn(n, E, device="cuda", generator=torch.Generator("cuda").manual_seed(73))
    kw, first = {}, 4
    if local < E:
        emap = torch.full((E,), -1, dtype=torch.int32, device="cuda")
        emap[first:first + local] = torch.arange(local, dtype=torch.int32, device="cuda")
        kw = dict(expert_map=emap, n_local_experts=local)
    p = moe.make_params(gating, "swiglu_oai", "interleaved", **kw)
    ws = moe.workspace_q4(n, E, k, H, I)
    indx = torch.empty(n, k, dtype=torch.int32, device="cuda")
    vals = torch.empty(n, k, dtype=BF16, device="cuda")
    meta = moe.empty_meta(n * k, local, "cuda")
    out = moe.forward_q4(x, z, w13, w2, k, p, ws, topk=(indx, vals), meta=meta)
    assert torch.equal(out, moe.forward_q4(x, z, w13, w2, k, p, ws))
    want_i, want_v = moe.route(z, k, gating)
    assert torch.equal(indx, want_i) and torch.equal(vals, want_v)
    y = moe.grouped_ffn_q4(x, meta, w13, w2, k, ws, p)
    assert torch.equal(out, moe.combine_weighted(y, meta, vals))
    assert moe.read_status(ws) == 0
    ref, tol = ffn64(x, meta, w13, w2, k, "swiglu_oai", "interleaved")
    row = meta["row_sorted"].long()
    live = row >= 0
    wt = torch.where(live, vals.double().reshape(-1), 0.0)[:, None]
    at = row.clamp_min(0)
    u = torch.finfo(BF16).eps / 2   # y's own rounding, then the sum's
    full = (wt * ref[at]).view(n, k, H).sum(1)
    err = (wt * (tol + u * (ref.abs() + tol) + 2.0 ** -134)[at]).view(n, k, H).sum(1)
    mag = (wt * ref[at].abs()).view(n, k, H).sum(1)
    check(out, full, err + 2 * (k + 1) * 2.0 ** -24 * mag)
