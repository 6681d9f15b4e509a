"""Rows to expert-sorted order and back (moe.dispatch, moe.combine_weighted),
their gradients, and the gate weights' gradient to the logits, against the
formulas in 64 bits.

Tolerances count roundings: u = eps / 2 of the row type for the one rounding
of a stored result, 2^-24 per fp32 operation of a sum (a sum of m products in
any order is off by at most (m + 1) 2^-24 times the sum of the magnitudes),
and half the row type's smallest subnormal below its normal range."""
import numpy as np
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe

pytestmark = pytest.mark.gpu

U32 = 2.0 ** -24
TINY = {torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25, torch.float32: 2.0 ** -150}
BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


def u(dtype):
    return torch.finfo(dtype).eps / 2


def make_meta(n, E, k, seed, local=None, dev="cuda"):
    """(topk_indx [n, k], meta over the `local` first experts) by explicit loops."""
    rng = np.random.default_rng(seed)
    indx = np.stack([rng.permutation(E)[:k] for _ in range(n)]).astype(np.int32) if n else \
        np.zeros((0, k), np.int32)
    local = E if local is None else local
    flat = indx.reshape(-1)
    col = [f for e in range(local) for f in np.nonzero(flat == e)[0]]
    row = np.full(n * k, -1, np.int32)
    for p, f in enumerate(col):
        row[f] = p
    offs = np.zeros(local + 1, np.int32)
    offs[1:] = np.cumsum([(flat == e).sum() for e in range(local)])
    t = lambda a: torch.from_numpy(np.ascontiguousarray(a)).to(dev)
    return t(indx), {"row_sorted": t(row), "offs": t(offs)}


def rows(shape, dtype, seed, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device="cuda") * scale).to(dtype)


def combine64(y, meta, w):
    n, k = w.shape
    row = meta["row_sorted"].long()
    live = (row >= 0) & (row < n * k)
    src = torch.where(live[:, None], y.double()[row.clamp(0, max(n * k - 1, 0))], 0.0)
    wf = torch.where(live, w.double().reshape(-1), 0.0)[:, None]
    H = y.shape[1]
    return (src * wf).view(n, k, H).sum(1), (src * wf).abs().view(n, k, H).sum(1), src, live


SIZES = [  # n, H, E, k, local
    (1, 2880, 32, 4, 32), (8, 2880, 32, 4, 32), (33, 64, 8, 2, 8), (33, 64, 8, 2, 3),
    (517, 1001, 16, 3, 8), (129, 1, 5, 5, 4), (64, 7, 12, 8, 12), (300, 130, 64, 7, 20),
    (4096, 512, 4, 1, 4), (257, 2056, 256, 8, 256), (70, 520, 16, 6, 1)]


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("n,H,E,k,local", SIZES)
def test_dispatch_and_its_gradient(n, H, E, k, local, dtype):
    _, meta = make_meta(n, E, k, 1, local)
    x = rows((n, H), dtype, 2)
    got = moe.dispatch(x, meta, k)
    row = meta["row_sorted"].long()
    want = torch.zeros(n * k, H, dtype=dtype, device="cuda")
    tok = torch.arange(n * k, device="cuda") // k
    want[row[row >= 0]] = x[tok[row >= 0]]
    assert torch.equal(got, want)

    d = rows((n * k, H), dtype, 3)
    got = moe.dispatch_backward(d, meta, k)
    ref, mag, _, _ = combine64(d, meta, torch.ones(n, k, device="cuda"))
    err = (got.double() - ref).abs()
    assert (err <= u(dtype) * ref.abs() * (1 + U32) + (k + 1) * U32 * mag + TINY[dtype]).all()


@pytest.mark.parametrize("wdtype", [BF16, FP32])
@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("n,H,E,k,local", SIZES)
def test_combine_and_its_gradients(n, H, E, k, local, dtype, wdtype):
    _, meta = make_meta(n, E, k, 4, local)
    y, d_out = rows((n * k, H), dtype, 5), rows((n, H), dtype, 6)
    w = torch.softmax(rows((n, k), FP32, 7), 1).to(wdtype)
    ref, mag, src, live = combine64(y, meta, w)
    got = moe.combine_weighted(y, meta, w)
    assert got.dtype == dtype
    err = (got.double() - ref).abs()
    assert (err <= u(dtype) * ref.abs() * (1 + U32) + 2 * (k + 1) * U32 * mag + TINY[dtype]).all()

    d_sorted, d_w = moe.combine_weighted_backward(d_out, y, meta, w)
    assert d_sorted.dtype == dtype and d_w.dtype == FP32
    up = d_out.double().repeat_interleave(k, 0)
    ref_w = (up * src).sum(1) * live
    mag_w = (up * src).abs().sum(1) * live
    assert ((d_w.double().reshape(-1) - ref_w).abs() <= (H + 1) * U32 * mag_w).all()
    assert (d_w.reshape(-1)[~live] == 0).all()
    row = meta["row_sorted"].long()
    ref_s = torch.zeros(n * k, H, dtype=torch.float64, device="cuda")
    ref_s[row[live]] = (w.double().reshape(-1, 1) * up)[live]
    err = (d_sorted.double() - ref_s).abs()
    assert (err <= (u(dtype) + 2 * U32) * ref_s.abs() + TINY[dtype]).all()


def test_gradients_against_differences():
    """dispatch and combine_weighted are linear in each argument, so a central
    difference of any width equals the derivative but for fp32 roundings:
    (m + 2) 2^-24 of the summed magnitudes on either side."""
    n, H, E, k, local = 40, 96, 8, 3, 6
    _, meta = make_meta(n, E, k, 8, local)
    y, v = rows((n * k, H), FP32, 9), rows((n * k, H), FP32, 10)
    d_out, w, dw = rows((n, H), FP32, 11), rows((n, k), FP32, 12), rows((n, k), FP32, 13)
    d_sorted, d_w = moe.combine_weighted_backward(d_out, y, meta, w)

    def loss(yy, ww):
        return (moe.combine_weighted(yy, meta, ww).double() * d_out.double()).sum().item()

    bound = 8 * (H + k + 2) * U32 * (d_out.double().abs().repeat_interleave(k, 0).sum() *
                                     max(y.abs().max(), v.abs().max()) *
                                     max(w.abs().max(), dw.abs().max())).item()
    num = (loss(y + v, w) - loss(y - v, w)) / 2
    assert abs(num - (d_sorted.double() * v.double()).sum().item()) <= bound
    num = (loss(y, w + dw) - loss(y, w - dw)) / 2
    assert abs(num - (d_w.double() * dw.double()).sum().item()) <= bound

    x, d_x = rows((n, H), FP32, 14), moe.dispatch_backward(v, meta, k)
    num = (moe.dispatch(x, meta, k).double() * v.double()).sum().item()
    assert abs(num - (d_x.double() * x.double()).sum().item()) <= bound


@pytest.mark.parametrize("n,E,k", [(1, 1, 1), (33, 8, 2), (5, 3, 3), (100, 32, 4), (77, 37, 5),
                                   (1000, 128, 4), (63, 130, 8), (64, 255, 7), (512, 256, 8)])
@pytest.mark.parametrize("gating", ["softmax_topk", "softmax_all"])
def test_route_backward(n, E, k, gating):
    z = rows((n, E), FP32, 20, 2.0)
    if E > 2 * k:   # masked experts among those not selected
        z[:, ::5] = float("-inf")
    indx, _ = moe.route(z, k, gating)
    d = rows((n, k), FP32, 21)
    got = moe.route_backward(z, indx, d, gating).double()
    zz, idx = z.double(), indx.long()
    chosen = torch.zeros(n, E, dtype=torch.bool, device="cuda").scatter_(1, idx, True)
    up = torch.zeros(n, E, dtype=torch.float64, device="cuda").scatter_(1, idx, d.double())
    if gating == "softmax_topk":
        zz = zz.masked_fill(~chosen, float("-inf"))
    p = torch.softmax(zz, 1)
    mean_mag = (p * up.abs()).sum(1, keepdim=True)
    ref = p * (up - (p * up).sum(1, keepdim=True))
    # a probability: the argument's subtraction, expf within 2 ulp (4 u), the
    # sum of at most E terms of the same kind, the division
    span = (zz.masked_fill(~zz.isfinite(), 0.0).abs().max() * 2).item()
    dp = (2 * (span + 4) + E + 4) * U32
    tol = p * (up.abs() + mean_mag) * (2 * dp + (k + 4) * U32) + 2.0 ** -140
    assert ((got - ref).abs() <= tol).all()
    # against differences of the gate weights in 64 bits, the selection fixed
    v = torch.randn(n, E, dtype=torch.float64, device="cuda")

    def vals(h):
        q = (zz + h * v).masked_fill(~zz.isfinite(), float("-inf"))
        return torch.gather(torch.softmax(q, 1), 1, idx)

    h = 1e-4   # truncation h^2 / 6 of a third derivative below 6 |v|^3; cancellation 2^-52 / h
    num = (((vals(h) - vals(-h)) / (2 * h)) * d.double()).sum(1)
    vmax = v.abs().max().item()
    slack = (h * h * (2 * vmax) ** 3 + 2.0 ** -50 / h) * d.double().abs().sum(1)
    assert ((num - (got * v).sum(1)).abs() <= slack + (tol * v.abs()).sum(1)).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
def test_bases_off_the_vector_width(dtype):
    """Rows that start one element into an allocation, where only narrow
    vectors are aligned, give the same bits."""
    n, H, k = 50, 256, 4
    _, meta = make_meta(n, 8, k, 30, 6)
    w = torch.softmax(rows((n, k), FP32, 31), 1)

    def off(t):
        buf = torch.empty(t.numel() + 1, dtype=t.dtype, device="cuda")
        v = buf[1:].view(t.shape)
        v.copy_(t)
        assert v.data_ptr() % 16 != 0
        return v

    x, y = rows((n, H), dtype, 32), rows((n * k, H), dtype, 33)
    assert torch.equal(moe.dispatch(off(x), meta, k), moe.dispatch(x, meta, k))
    assert torch.equal(moe.dispatch(x, meta, k, out=off(y)), moe.dispatch(x, meta, k))
    assert torch.equal(moe.combine_weighted(off(y), meta, w), moe.combine_weighted(y, meta, w))
    a = moe.combine_weighted_backward(off(x), off(y), meta, w)
    b = moe.combine_weighted_backward(x, y, meta, w)
    assert torch.equal(a[0], b[0])
    # another vector width adds the products in another order
    mag = x.double().abs().repeat_interleave(k, 0).max() * y.double().abs().max()
    assert ((a[1] - b[1]).abs() <= 2 * (H + 1) * U32 * H * mag).all()


class Guarded:
    """An array `off` elements past a 16-byte boundary, ones of 7 before and after it."""

    def __init__(self, shape, dtype, off):
        size = int(np.prod(shape))
        self.buf = torch.full((size + 64,), 7.0, dtype=dtype, device="cuda")
        self.lo, self.hi = 16 + off, 16 + off + size
        self.t = self.buf[self.lo:self.hi].view(shape)

    def untouched(self):
        return bool((self.buf[:self.lo] == 7).all() and (self.buf[self.hi:] == 7).all())


def surrounded(t, off):
    """A copy of t at such a place, between NaN."""
    g = Guarded(t.shape, t.dtype, off)
    g.buf.fill_(float("nan"))
    g.t.copy_(t)
    return g.t


@pytest.mark.parametrize("dtype", [BF16, FP16, FP32])
@pytest.mark.parametrize("H", [1, 2, 3, 4, 7, 9, 12, 31, 255, 1442, 4099, 8200])
@pytest.mark.parametrize("k", [1, 2, 4, 7])
def test_rows_at_every_alignment(H, dtype, k):
    """Rows and arrays that start anywhere: what lies around an array is
    neither used nor written, and copies and scaled copies have their exact
    bits (one product in fp32, one rounding)."""
    n, E, per = 13, 9, 16 // torch.finfo(dtype).bits * 8
    _, meta = make_meta(n, E, k, 50, 6)
    row, kept = meta["row_sorted"].long(), int(meta["offs"][-1])
    x, y, d_out = rows((n, H), dtype, 51), rows((n * k, H), dtype, 52), rows((n, H), dtype, 53)
    y[kept:] = float("nan")
    w = torch.softmax(rows((n, k), FP32, 54), 1)
    live = row >= 0
    token = torch.arange(n, device="cuda").repeat_interleave(k)[live]
    want = torch.zeros(n * k, H, dtype=dtype, device="cuda")
    want[row[live]] = x[token]
    scaled = torch.zeros_like(want)
    scaled[row[live]] = (w.reshape(-1, 1)[live] * d_out[token].float()).to(dtype)
    ref, mag, src, _ = combine64(torch.where(torch.isnan(y), 0.0, y), meta, w)
    up = d_out.double().repeat_interleave(k, 0)
    ref_w, mag_w = (up * src).sum(1) * live, (up * src).abs().sum(1) * live
    for a, b, c in [(0, 0, 0), (1, 0, 0), (0, 1, 0), (0, 0, 1), (1, 1, 1), (3, 2, 1),
                    (per - 1, 1, per - 1), (2, per - 1, 2)]:
        g = Guarded((n * k, H), dtype, b)
        moe.dispatch(surrounded(x, a), meta, k, out=g.t)
        assert g.untouched() and torch.equal(g.t, want)

        yy, g = surrounded(y, a), Guarded((n, H), dtype, b)
        moe.combine_weighted(yy, meta, w, out=g.t)
        err = (g.t.double() - ref).abs()
        assert g.untouched()
        assert (err <= u(dtype) * ref.abs() * (1 + U32) + 2 * (k + 1) * U32 * mag +
                TINY[dtype]).all()

        g, d_w = Guarded((n * k, H), dtype, c), torch.empty(n, k, device="cuda")
        code = {BF16: 0, FP16: 1, FP32: 2}
        moe._binding._run("moe_combine_weighted_backward", 0, surrounded(d_out, b).data_ptr(),
                          yy.data_ptr(), meta["row_sorted"].data_ptr(), w.data_ptr(), code[FP32],
                          moe._binding._kept(meta), n, k, H, code[dtype], g.t.data_ptr(),
                          d_w.data_ptr())
        assert g.untouched() and torch.equal(g.t, scaled)
        assert ((d_w.double().reshape(-1) - ref_w).abs() <= (H + 1) * U32 * mag_w).all()


@pytest.mark.parametrize("dtype", [BF16, FP32])
@pytest.mark.parametrize("n,k,local", [(2047, 1, 5), (2051, 1, 5), (2049, 2, 6), (5001, 2, 8),
                                       (4097, 1, 8)])
def test_many_tokens_of_one_or_two_slots(n, k, local, dtype):
    """Several tokens share a thread here; the last ones are no full group."""
    H, E = 264, 8
    _, meta = make_meta(n, E, k, 55, local)
    y, w = rows((n * k, H), dtype, 56), rows((n, k), FP32, 57)
    y[int(meta["offs"][-1]):] = float("nan")
    ref, mag, _, _ = combine64(torch.where(torch.isnan(y), 0.0, y), meta, w)
    g = Guarded((n, H), dtype, 0)
    moe.combine_weighted(y, meta, w, out=g.t)
    assert g.untouched()
    err = (g.t.double() - ref).abs()
    assert (err <= u(dtype) * ref.abs() * (1 + U32) + 2 * (k + 1) * U32 * mag + TINY[dtype]).all()
    ref, mag, _, _ = combine64(torch.where(torch.isnan(y), 0.0, y), meta, torch.ones_like(w))
    err = (moe.dispatch_backward(y, meta, k).double() - ref).abs()
    assert (err <= u(dtype) * ref.abs() * (1 + U32) + 2 * (k + 1) * U32 * mag + TINY[dtype]).all()


def test_dropped_slots_are_not_read():
    """A dropped slot (-1, or an index past the rows) adds nothing even where
    its weight is NaN; a token without a kept slot gets zeros; rows past the
    kept ones stay out of every sum."""
    n, H, k = 6, 64, 2
    N = n * k
    row = torch.full((N,), -1, dtype=torch.int32)
    row[[0, 3, 4]] = torch.tensor([2, 0, 1], dtype=torch.int32)
    row[5], row[6], row[7] = N, 2 ** 31 - 1, -(2 ** 31)
    meta = {"row_sorted": row.cuda(), "offs": torch.tensor([0, 2, 3], dtype=torch.int32).cuda()}
    y = rows((N, H), BF16, 40)
    y[3:] = float("nan")
    w = torch.rand(n, k, device="cuda")
    w.view(-1)[row.cuda() < 0] = float("nan")
    w.view(-1)[5:7] = float("inf")
    out = moe.combine_weighted(y, meta, w)
    ref, mag, _, live = combine64(y, {"row_sorted": torch.where(
        (row >= 0) & (row < N), row, -1).cuda()}, w)
    assert out.isfinite().all() and (out[3:] == 0).all()
    assert ((out.double() - ref).abs() <= u(BF16) * ref.abs() * (1 + U32) + 6 * U32 * mag).all()
    x = rows((n, H), BF16, 41)
    sorted_x = moe.dispatch(x, meta, k)
    assert torch.equal(sorted_x[[2, 0, 1]], x[[0, 1, 2]]) and (sorted_x[3:] == 0).all()
    ds, dw = moe.combine_weighted_backward(x, y, meta, w)
    assert ds.isfinite().all() and dw.isfinite().all() and (ds[3:] == 0).all()
    assert (dw.view(-1)[[1, 2, 5, 6, 7, 8, 9, 10, 11]] == 0).all()
    none = {"row_sorted": torch.full((N,), -1, dtype=torch.int32, device="cuda"),
            "offs": torch.zeros(2, dtype=torch.int32, device="cuda")}
    assert (moe.combine_weighted(y, none, w) == 0).all()
    assert (moe.dispatch(x, none, k) == 0).all()
    assert (moe.dispatch_backward(y, none, k) == 0).all()


def test_kept_values_pass_through_unchanged():
    """Infinities and NaN in kept rows reach the outputs that they belong to
    and no others."""
    n, H, k = 4, 72, 1
    _, meta = make_meta(n, 3, k, 50)
    x = rows((n, H), FP16, 51)
    x[1, 5], x[2, 70] = float("inf"), float("nan")
    y = moe.dispatch(x, meta, k)
    out = moe.combine_weighted(y, meta, torch.ones(n, k, device="cuda"))
    torch.testing.assert_close(out, x, rtol=0, atol=0, equal_nan=True)


def test_no_tokens():
    meta = {"row_sorted": torch.empty(0, dtype=torch.int32, device="cuda"),
            "offs": torch.zeros(5, dtype=torch.int32, device="cuda")}
    x = torch.empty(0, 64, dtype=BF16, device="cuda")
    w = torch.empty(0, 2, device="cuda")
    assert moe.dispatch(x, meta, 2).shape == (0, 64)
    assert moe.dispatch_backward(x, meta, 2).shape == (0, 64)
    assert moe.combine_weighted(x, meta, w).shape == (0, 64)
    ds, dw = moe.combine_weighted_backward(x, x, meta, w)
    assert ds.shape == (0, 64) and dw.shape == (0, 2)
    z = torch.empty(0, 8, device="cuda")
    assert moe.route_backward(z, torch.empty(0, 2, dtype=torch.int32, device="cuda"),
                              torch.empty(0, 2, device="cuda")).shape == (0, 8)


def test_offsets_past_32_bits():
    """More than 2^32 bytes and 2^31 elements of sorted rows."""
    n, H, k = 300_000, 1920, 4
    N = n * k
    row = torch.arange(N - 1, -1, -1, dtype=torch.int32, device="cuda")
    meta = {"row_sorted": row, "offs": torch.tensor([0, N], dtype=torch.int32, device="cuda")}
    x = (torch.arange(n, device="cuda") % 251).to(BF16)[:, None].expand(n, H).contiguous()
    s = moe.dispatch(x, meta, k)
    tok = (N - 1 - torch.arange(N, device="cuda")) // k
    assert torch.equal(s[:, 0], x[tok, 0]) and torch.equal(s[:, -1], x[tok, 0])
    w = torch.full((n, k), 0.25, device="cuda")
    assert torch.equal(moe.combine_weighted(s, meta, w), x)
    ds, dw = moe.combine_weighted_backward(x, s, meta, w)
    assert torch.equal(ds[:, 7], x[tok, 0] * 0.25) and torch.equal(ds[:, -1], x[tok, 0] * 0.25)
    want = x[:, 0].double() ** 2 * H   # whole numbers; the rounded sums stay within H 2^-24
    assert ((dw.double() - want[:, None]).abs() <= H * U32 * want[:, None]).all()


def test_other_streams_and_repeats():
    """On a side stream, and twice on one input: the same bits."""
    n, H, k = 700, 2880, 4
    _, meta = make_meta(n, 32, k, 60, 20)
    x, y = rows((n, H), BF16, 61), rows((n * k, H), BF16, 62)
    w = torch.softmax(rows((n, k), FP32, 63), 1)

    def every():
        return [moe.dispatch(x, meta, k), moe.dispatch_backward(y, meta, k),
                moe.combine_weighted(y, meta, w), *moe.combine_weighted_backward(x, y, meta, w)]

    first = every()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        second = every()
    torch.cuda.current_stream().wait_stream(side)
    for a, b in zip(first, second):
        assert torch.equal(a, b)


def test_graph_capture():
    n, H, k = 96, 520, 4
    _, meta = make_meta(n, 16, k, 70, 9)
    x, y = rows((n, H), BF16, 71), rows((n * k, H), BF16, 72)
    z = rows((n, 16), FP32, 73)
    indx, vals = moe.route(z, k)
    moe.dispatch(x, meta, k)   # first calls before the capture
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        s = moe.dispatch(x, meta, k)
        out = moe.combine_weighted(y, meta, vals)
        ds, dw = moe.combine_weighted_backward(x, y, meta, vals)
        dx = moe.dispatch_backward(ds, meta, k)
        dz = moe.route_backward(z, indx, dw)
    x.copy_(rows((n, H), BF16, 74))
    y.copy_(rows((n * k, H), BF16, 75))
    graph.replay()
    ds2, dw2 = moe.combine_weighted_backward(x, y, meta, vals)
    for a, b in ((s, moe.dispatch(x, meta, k)), (out, moe.combine_weighted(y, meta, vals)),
                 (ds, ds2), (dw, dw2), (dx, moe.dispatch_backward(ds2, meta, k)),
                 (dz, moe.route_backward(z, indx, dw2))):
        assert torch.equal(a, b)


def test_with_the_layers_own_metadata():
    """route_metadata -> dispatch -> (identity experts) -> combine_weighted
    gives x times the sum of the gate weights; and an expert map's metadata
    from moe.forward drops the slots of the other experts."""
    n, H, E, k, I = 200, 128, 16, 4, 64
    z, x = rows((n, E), FP32, 80), rows((n, H), BF16, 81)
    indx, vals, meta = moe.route_metadata(z, k)
    s = moe.dispatch(x, meta, k)
    order = meta["col_sorted"].long() // k
    assert torch.equal(s, x[order])
    out = moe.combine_weighted(s, meta, vals)
    ref, mag, _, _ = combine64(s, meta, vals)
    err = (out.double() - ref).abs()
    assert (err <= u(BF16) * ref.abs() * (1 + U32) + 2 * (k + 1) * U32 * mag).all()

    local = 5
    emap = torch.full((E,), -1, dtype=torch.int32, device="cuda")
    emap[3:3 + local] = torch.arange(local, dtype=torch.int32, device="cuda")
    p = moe.make_params(expert_map=emap, n_local_experts=local)
    w13, w2 = rows((local, 2 * I, H), BF16, 82, 0.05), rows((local, H, I), BF16, 83, 0.05)
    m = moe.empty_meta(n * k, local, "cuda")
    ws = moe.workspace(n, E, k, H, I)
    moe.forward(x, z, w13, w2, k, p, ws, meta=m)
    s = moe.dispatch(x, m, k)
    kept = int(m["offs"][-1])
    assert 0 < kept < n * k
    assert torch.equal(s[:kept], x[m["col_sorted"][:kept].long() // k])
    assert (s[kept:] == 0).all()
