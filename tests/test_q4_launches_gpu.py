"""The launches that the experts' 4-bit products take for long rows, for two
formats and for the layer (moe.grouped_ffn_q4, moe.forward_q4), in every format
and type."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from test_q4_experts_gpu import experts64, weights
from test_q4_gpu import BF16, FP16, check, make_meta, random_q4, tokens

pytestmark = pytest.mark.gpu

# n, H, I: rows up to 3712 columns (29 slabs of 128) have room for two token
# blocks, up to about 8000 for one; longer ones come in chunks. Two experts and
# one slot per token.
LAUNCHES = [(3, 3776, 192), (40, 3776, 192), (3, 192, 3776), (40, 192, 3776), (40, 3776, 3776),
            (1, 8320, 64), (40, 8320, 64), (1, 64, 8320), (40, 64, 8320), (40, 3840, 8320),
            (40, 8320, 3840)]


@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("n,H,I", LAUNCHES)
def test_rows_too_long_for_one_launch(n, H, I, fmt):
    E, k = 2, 1
    w13, w2 = weights(fmt, E, H, I, "swiglu", 130)
    meta, x = make_meta(n, E, k, 132), tokens(n, H, BF16 if n > 1 else FP16, 133, 0.1)
    ws = moe.workspace_q4(n, E, k, H, I)
    got = moe.grouped_ffn_q4(x, meta, w13, w2, k, ws, moe.make_params())
    check(got, *experts64(x, meta, w13, w2, k, "swiglu", "packed"))
    assert moe.read_status(ws) == 0


@pytest.mark.parametrize("formats", [("mxfp4", "nvfp4"), ("nvfp4", "mxfp4")])
@pytest.mark.parametrize("n,H,I", [(2, 256, 192), (60, 256, 192), (60, 128, 8320), (60, 8320, 128)])
def test_two_formats_at_every_launch(n, H, I, formats):
    E, k = 3, 2
    w13 = random_q4((2 * I, H), formats[0], 140, count=E)
    w2 = random_q4((H, I), formats[1], 141, count=E)
    meta, x = make_meta(n, E, k, 142), tokens(n, H, BF16, 143, 0.1)
    got = moe.grouped_ffn_q4(x, meta, w13, w2, k, moe.workspace_q4(n, E, k, H, I),
                             moe.make_params())
    check(got, *experts64(x, meta, w13, w2, k, "swiglu", "packed"))


@pytest.mark.parametrize("n,H,I", [(24, 3776, 192), (24, 64, 8320), (24, 256, 192)])
def test_layer_in_a_graph(n, H, I):
    """Every launch of the layer in a graph, on new inputs, and repeated."""
    E, k = 4, 2
    w13, w2 = weights("mxfp4", E, H, I, "swiglu", 150)
    p, ws = moe.make_params(), moe.workspace_q4(n, E, k, H, I)
    x, z = tokens(n, H, BF16, 152, 0.1), torch.randn(n, E, device="cuda")
    moe.forward_q4(x, z, w13, w2, k, p, ws)
    torch.cuda.synchronize()
    graph, out = torch.cuda.CUDAGraph(), torch.empty_like(x)
    with torch.cuda.graph(graph):
        moe.forward_q4(x, z, w13, w2, k, p, ws, out=out)
    for seed in (153, 154):
        x.copy_(tokens(n, H, BF16, seed, 0.1))
        z.copy_(torch.randn(n, E, device="cuda"))
        graph.replay()
        first = out.clone()
        graph.replay()
        assert torch.equal(out, first)
        assert torch.equal(out, moe.forward_q4(x, z, w13, w2, k, p, ws))
    assert moe.read_status(ws) == 0


@pytest.mark.parametrize("dtype", [BF16, FP16])
@pytest.mark.parametrize("fmt", ["mxfp4", "nvfp4"])
@pytest.mark.parametrize("n,E,k,local", [(1, 8, 2, 8), (13, 8, 3, 2), (300, 16, 4, 16),
                                         (2, 1, 1, 1), (160000, 8, 8, 8)])
def test_layer_in_every_format_and_type(n, E, k, local, fmt, dtype):
    """forward_q4 against its stages and the formula; the last size is past
    what the one routing kernel takes."""
    H, I = 64, 64
    w13, w2 = weights(fmt, local, H, I, "swiglu_oai", 160)
    x = tokens(n, H, dtype, 162)
    z = torch.randn(n, E, device="cuda", generator=torch.Generator("cuda").manual_seed(163))
    kw = {}
    if local < E:
        emap = torch.full((E,), -1, dtype=torch.int32, device="cuda")
        emap[1:1 + local] = torch.arange(local, dtype=torch.int32, device="cuda")
        kw = dict(expert_map=emap, n_local_experts=local)
    p = moe.make_params("softmax_topk", "swiglu_oai", "interleaved", **kw)
    ws = moe.workspace_q4(n, E, k, H, I)
    vals = torch.empty(n, k, dtype=BF16, device="cuda")
    indx = torch.empty(n, k, dtype=torch.int32, device="cuda")
    meta = moe.empty_meta(n * k, local, "cuda")
    out = moe.forward_q4(x, z, w13, w2, k, p, ws, topk=(indx, vals), meta=meta)
    y = moe.grouped_ffn_q4(x, meta, w13, w2, k, ws, p)
    assert moe.read_status(ws) == 0
    ref, tol = experts64(x, meta, w13, w2, k, "swiglu_oai", "interleaved")
    check(y, ref, tol)
    row = meta["row_sorted"].long()
    live, at = row >= 0, row.clamp_min(0)
    wt = torch.where(live, vals.double().reshape(-1), 0.0)[:, None]
    src = y.double()[at]           # the layer's own rows: only its sum is left to bound
    full, mag = (wt * src).view(n, k, H).sum(1), (wt * src.abs()).view(n, k, H).sum(1)
    check(out, full, 2 * (k + 1) * 2.0 ** -24 * mag)
