"""How the calls of the dense blocks may be made: on any stream, captured into a
graph and replayed, two at a time, with buffers of the caller's, at any place
in memory; rows behind the last stay as they were; and what the binding refuses."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import Gate, act_slack, check, halves, mx8_rows, product, randn

pytestmark = pytest.mark.gpu


def gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


class Block:
    """Inputs of every call, and the calls by name."""

    def __init__(self, n, H, I, seed=0):
        g = gen(seed)
        self.x, self.res, self.d_y = (randn(g, n, H) for _ in range(3))
        self.d_h, self.h = randn(g, n, I), randn(g, n, I)
        self.w = 1 + 0.1 * randn(g, H, dtype=torch.float32)
        self.w13, self.w2 = randn(g, 2 * I, H, scale=H ** -0.5), randn(g, H, I, scale=I ** -0.5)
        self.bias = randn(g, H)
        self.x8 = moe.Mx8(*mx8_rows(g, n, H))
        self.h8 = moe.Mx8(*mx8_rows(g, n, I))
        self.w13_8 = moe.Mx8(*mx8_rows(g, 2 * I, H, H ** -0.5))
        self.w2_8 = moe.Mx8(*mx8_rows(g, H, I, I ** -0.5))
        self.params = moe.make_params(act="swiglu_oai", layout="packed")

    def calls(self):
        return {
            "norm": lambda: moe.rms_norm(self.x, self.w, residual=self.res),
            "norm8": lambda: moe.rms_norm(self.x, self.w, mx8=True),
            "norm_grad": lambda: moe.rms_norm_backward(self.d_y, self.x, self.w, d_sum=self.res),
            "linear": lambda: moe.linear(self.h, self.w2, self.bias, "gelu", self.res),
            "linear8": lambda: moe.linear(self.h8, self.w2_8, self.bias, "none", self.res),
            "linear_grad": lambda: moe.linear_backward(self.d_y, self.h, self.w2, self.bias,
                                                       "silu"),
            "linear_grad_none": lambda: moe.linear_backward(self.d_y, self.h, self.w2, self.bias),
            "gated": lambda: moe.gated_linear(self.x, self.w13, self.params),
            "gated8": lambda: moe.gated_linear(self.x8, self.w13_8, self.params, mx8=True),
            "gated_grad": lambda: moe.gated_linear_backward(self.d_h, self.x, self.w13,
                                                            self.params)}


def flat(out):
    if isinstance(out, moe.Mx8):
        return [out.codes.view(torch.uint8), out.scales]
    return [t for o in (out if isinstance(out, tuple) else (out,)) if o is not None
            for t in (flat(o) if isinstance(o, moe.Mx8) else [o])]


def same(a, b):
    return all(torch.equal(x, y) for x, y in zip(flat(a), flat(b)))


SIZES = [(3, 64, 96), (40, 2880, 96), (300, 512, 1408)]


@pytest.mark.parametrize("n,H,I", SIZES)
def test_the_same_bits_again_and_on_another_stream(n, H, I):
    b = Block(n, H, I)
    side = torch.cuda.Stream()
    for name, fn in b.calls().items():
        first = fn()
        assert same(first, fn()), name
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            other = fn()
        torch.cuda.current_stream().wait_stream(side)
        assert same(first, other), name


@pytest.mark.parametrize("n,H,I", SIZES)
def test_captured_and_replayed_on_new_inputs(n, H, I):
    b, other = Block(n, H, I, 1), Block(n, H, I, 2)
    for name in b.calls():
        work = Block(n, H, I, 1)
        fn = work.calls()[name]
        fn()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = fn()
        for src in (b, other, b):
            for k, v in vars(src).items():
                mine = getattr(work, k)
                if isinstance(v, torch.Tensor):
                    mine.copy_(v)
                elif isinstance(v, moe.Mx8):
                    mine.codes.view(torch.uint8).copy_(v.codes.view(torch.uint8))
                    mine.scales.copy_(v.scales)
            graph.replay()
            assert same(src.calls()[name](), out), name


def test_two_graphs_and_an_eager_call_at_a_time():
    """Each call has scratch of its own: two captured graphs that replay on two
    streams while a third call runs."""
    b, c = Block(200, 256, 1024, 1), Block(200, 256, 1024, 2)
    for name in b.calls():
        fb, fc = b.calls()[name], c.calls()[name]
        want_b, want_c = fb(), fc()
        torch.cuda.synchronize()
        gb, gc = torch.cuda.CUDAGraph(), torch.cuda.CUDAGraph()
        with torch.cuda.graph(gb):
            for _ in range(8):
                out_b = fb()
        with torch.cuda.graph(gc):
            for _ in range(8):
                out_c = fc()
        s1, s2 = torch.cuda.Stream(), torch.cuda.Stream()
        for s in (s1, s2):
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            with torch.cuda.stream(s1):
                gb.replay()
            with torch.cuda.stream(s2):
                gc.replay()
            eager = fb()
            torch.cuda.synchronize()
            assert same(want_b, out_b) and same(want_c, out_c) and same(want_b, eager), name


def test_two_host_threads():
    """Two threads call at once, on one stream and on two."""
    import threading

    b, c = Block(90, 256, 512, 1), Block(90, 256, 512, 2)
    want = [{k: fn() for k, fn in x.calls().items()} for x in (b, c)]
    torch.cuda.synchronize()
    for streams in ([None, None], [torch.cuda.Stream(), torch.cuda.Stream()]):
        bad = []

        def work(i):
            with torch.cuda.stream(streams[i]):
                for _ in range(10):
                    got = {k: fn() for k, fn in (b, c)[i].calls().items()}
                    torch.cuda.current_stream().synchronize()
                    bad.extend(k for k in got if not same(want[i][k], got[k]))

        threads = [threading.Thread(target=work, args=(i,)) for i in range(2)]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        assert not bad, bad


def test_buffers_of_the_callers():
    b = Block(130, 512, 1024, 3)
    n, H = b.x.shape
    I = b.h.shape[1]
    st = torch.zeros(1, dtype=torch.int32, device="cuda")

    def ws(size):
        return torch.full((max(size, 1),), 0xA5, dtype=torch.uint8, device="cuda")

    want, got = moe.linear(b.h, b.w2, b.bias), torch.empty_like(b.x)
    assert moe.linear(b.h, b.w2, b.bias, out=got, ws=ws(moe.linear_workspace_size(n, H, I)),
                      status=st) is got
    assert same(want, got)
    assert same(moe.linear(b.h8, b.w2_8),
                moe.linear(b.h8, b.w2_8, ws=ws(moe.linear_workspace_size(n, H, I, True))))
    assert same(moe.gated_linear(b.x, b.w13, b.params),
                moe.gated_linear(b.x, b.w13, b.params, status=st,
                                 ws=ws(moe.gated_linear_workspace_size(n, H, I))))
    q = moe.Mx8(torch.empty_like(b.h8.codes), torch.empty_like(b.h8.scales))
    assert moe.gated_linear(b.x8, b.w13_8, b.params, mx8=True, out=q) is q
    assert same(moe.gated_linear(b.x8, b.w13_8, b.params, mx8=True), q)
    assert same(moe.linear_backward(b.d_y, b.h, b.w2, b.bias, "silu"),
                moe.linear_backward(b.d_y, b.h, b.w2, b.bias, "silu", status=st,
                                    ws=ws(moe.linear_backward_workspace_size(n, H, I, "silu"))))
    assert same(moe.gated_linear_backward(b.d_h, b.x, b.w13, b.params),
                moe.gated_linear_backward(
                    b.d_h, b.x, b.w13, b.params, status=st,
                    ws=ws(moe.gated_linear_backward_workspace_size(n, H, I))))
    assert same(moe.rms_norm_backward(b.d_y, b.x, b.w),
                moe.rms_norm_backward(b.d_y, b.x, b.w,
                                      ws=ws(moe.rms_norm_backward_workspace_size(n, H))))
    y, s = moe.rms_norm(b.x, b.w, residual=b.res)
    o, t = torch.empty_like(b.x), torch.empty_like(b.x)
    assert moe.rms_norm(b.x, b.w, residual=b.res, out=o, sum_out=t)[0] is o
    assert same((y, s), (o, t))
    assert st.item() == 0


@pytest.mark.parametrize("n", [1, 20, 33, 129, 300])
@pytest.mark.parametrize("R", [40, 77, 1000])
def test_nothing_behind_the_last_row_or_beside_it(n, R):
    """Outputs between guards, and inputs whose rows behind the last are NaN."""
    g = gen(n + R)
    C = 136
    big = randn(g, n + 40, C)
    big[n:] = float("nan")
    w = torch.full((R + 20, C), float("nan"), dtype=torch.bfloat16, device="cuda")
    w[:R] = randn(g, R, C, scale=C ** -0.5)
    buf = torch.full((8 + n * R + 300,), 3.0, dtype=torch.bfloat16, device="cuda")
    for off in (0, 8, 1):                      # rows on 16 bytes, and not
        buf.fill_(3.0)
        out = buf[off:off + n * R].view(n, R)
        res = randn(g, n * R + 1)[1:].view(n, R)   # off 16 bytes itself
        bias = randn(g, R + 1)[1:]
        moe.linear(big[:n], w[:R], bias=bias, act="silu", residual=res, out=out)
        a, da = product(big[:n], w[:R])
        a, da = a + bias.double(), da + 2.0 ** -23 * (a.abs() + bias.double().abs())
        y = a * torch.sigmoid(a)
        check(out, y + res.double(),
              act_slack(a, da, "silu") + 2.0 ** -23 * (y.abs() + res.double().abs()))
        assert (buf[:off] == 3).all() and (buf[off + n * R:] == 3).all()


@pytest.mark.parametrize("n", [5, 33, 200])
def test_gated_between_guards(n):
    g = gen(n)
    H, I = 72, 48
    x, w = randn(g, n, H), randn(g, 2 * I, H, scale=H ** -0.5)
    params = moe.make_params(act="swiglu", layout="packed")
    buf = torch.full((n * I + 64,), 3.0, dtype=torch.bfloat16, device="cuda")
    a, da = product(x, w)
    (p, u), (dp, du) = halves(a, "packed"), halves(da, "packed")
    h, slack = Gate("swiglu").forward(p, u, dp, du)
    for off in (0, 1):                         # a result off 16 bytes
        buf.fill_(3.0)
        out = buf[off:off + n * I].view(n, I)
        moe.gated_linear(x, w, params, out=out)
        check(out, h, slack)
        assert (buf[:off] == 3).all() and (buf[off + n * I:] == 3).all()
    d_h = randn(g, n * I + 1)[1:].view(n, I)   # a gradient off 16 bytes
    assert same(moe.gated_linear_backward(d_h, x, w, params),
                moe.gated_linear_backward(d_h.clone(), x, w, params))


def test_no_rows():
    b = Block(0, 64, 96)
    y, s = moe.rms_norm(b.x, b.w, residual=b.res)
    assert y.shape == s.shape == (0, 64)
    assert moe.linear(b.h, b.w2).shape == (0, 64)
    assert moe.linear(b.h8, b.w2_8).shape == (0, 64)
    assert moe.gated_linear(b.x, b.w13, b.params).shape == (0, 96)
    d_x, d_w, d_bias = moe.linear_backward(b.d_y, b.h, b.w2, b.bias, "silu")
    assert d_x.shape == (0, 96) and (d_w == 0).all() and (d_bias == 0).all()
    d_x, d_w = moe.gated_linear_backward(b.d_h, b.x, b.w13, b.params)
    assert (d_w == 0).all()
    d_x, d_w = moe.rms_norm_backward(b.d_y, b.x, b.w)
    assert (d_w == 0).all()


def test_gradients_that_are_not_wanted():
    """The C calls leave out what is NULL."""
    b = Block(70, 64, 96, 4)
    L, n, H, I = moe.lib(), 70, 64, 96
    full = moe.linear_backward(b.d_y, b.h, b.w2, b.bias, "silu")
    ws = torch.empty(moe.linear_backward_workspace_size(n, H, I, "silu"), dtype=torch.uint8,
                     device="cuda")
    s = torch.cuda.current_stream().cuda_stream
    for keep in range(8):
        got = [torch.full_like(t, 9.0) for t in full]
        ptr = [t.data_ptr() if keep >> i & 1 else None for i, t in enumerate(got)]
        assert L.moe_linear_backward(b.d_y.data_ptr(), b.h.data_ptr(), b.w2.data_ptr(),
                                     b.bias.data_ptr(), n, H, I, 0, 1, *ptr, ws.data_ptr(),
                                     ws.numel(), None, s) == 0
        torch.cuda.synchronize()
        for i, t in enumerate(got):
            assert torch.equal(t, full[i]) if keep >> i & 1 else (t == 9).all(), (keep, i)
    p = b.params
    import ctypes
    ws = torch.empty(moe.gated_linear_backward_workspace_size(n, H, I), dtype=torch.uint8,
                     device="cuda")
    full = moe.gated_linear_backward(b.d_h, b.x, b.w13, p)
    for keep in range(4):
        got = [torch.full_like(t, 9.0) for t in full]
        ptr = [t.data_ptr() if keep >> i & 1 else None for i, t in enumerate(got)]
        assert L.moe_gated_linear_backward(b.d_h.data_ptr(), b.x.data_ptr(), b.w13.data_ptr(), n,
                                           H, I, ctypes.byref(p), 0, *ptr, ws.data_ptr(),
                                           ws.numel(), None, s) == 0
        torch.cuda.synchronize()
        for i, t in enumerate(got):
            assert torch.equal(t, full[i]) if keep >> i & 1 else (t == 9).all(), (keep, i)


def test_binding_refuses():
    b = Block(4, 64, 96)
    for fn, match in (
            (lambda: moe.linear(b.x, b.w2), "shape"),
            (lambda: moe.linear(b.x, b.w13.half()), "bfloat16"),
            (lambda: moe.linear(b.x.t(), b.w13), "contiguous"),
            (lambda: moe.linear(b.x, b.w13.cpu()), "CUDA"),
            (lambda: moe.linear(b.x, b.w13, dtype=torch.float16), "x's"),
            (lambda: moe.linear(b.x8, b.w13), "Mx8"),
            (lambda: moe.linear(b.x, b.w13_8), "CUDA tensor"),
            (lambda: moe.linear(b.x8, b.w2_8), "columns"),
            (lambda: moe.linear(b.x8, b.w13_8, dtype=torch.float32), "bfloat16"),
            (lambda: moe.linear(b.x, b.w13, bias=b.bias), "shape"),
            (lambda: moe.linear(b.x, b.w13, residual=b.x), "shape"),
            (lambda: moe.linear(b.x, b.w13, out=b.x), "shape"),
            (lambda: moe.linear(b.x, b.w13, status=b.bias), "int32"),
            (lambda: moe.gated_linear(b.x, b.w13[:3], b.params), "even"),
            (lambda: moe.gated_linear(b.x, b.w13, b.params, mx8=True, out=b.h), "Mx8"),
            (lambda: moe.gated_linear(b.x, b.w13[:80].contiguous(), b.params, mx8=True), "32"),
            (lambda: moe.gated_linear_backward(b.x, b.x, b.w13, b.params), "shape"),
            (lambda: moe.linear_backward(b.x, b.x, b.w13), "shape"),
            (lambda: moe.rms_norm(b.x, b.w.double()), "weight"),
            (lambda: moe.rms_norm(b.x, b.w, sum_out=b.x), "residual"),
            (lambda: moe.rms_norm(b.x[:, :40].contiguous(), None, mx8=True), "32"),
            (lambda: moe.rms_norm_backward(b.d_h, b.x, b.w), "shape"),
            (lambda: moe.Mx8(b.x8.codes, b.x8.scales[:2].contiguous()), "shape"),
            (lambda: moe.Mx8(b.x8.codes.view(torch.uint8), b.x8.scales), "float8")):
        with pytest.raises(ValueError, match=match):
            fn()
    with pytest.raises(moe.MoEError, match="UNSUPPORTED"):
        moe.gated_linear(b.x, b.w13, moe.make_params(act="relu2"))
    small = torch.empty(16, dtype=torch.uint8, device="cuda")
    with pytest.raises(moe.MoEError, match="WORKSPACE"):
        moe.rms_norm_backward(b.d_y, b.x, b.w, ws=small)
    with pytest.raises(moe.MoEError, match="INVALID"):
        moe.linear(b.x[:, :60].contiguous(), b.w13[:, :60].contiguous())
