"""MXFP8 products over the whole range of scale bytes, 0 to 254: wherever the
product of two scales and their values is representable it comes out, however
far apart the two scales are, with few rows and with many."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from dense_reference import mx8_value

pytestmark = pytest.mark.gpu

ONE = 0x38                     # 1.0 as E4M3
TOP = 0x7e                     # 448, the largest
TINY = 0x01                    # 2^-9, the least
ROWS = [1, 8, 16, 40, 255]     # both kernels; 8 and 9 rows are a border


def rows8(codes, scales):
    return moe.Mx8(codes.view(torch.float8_e4m3fn), scales)


def token_bytes(n):
    """n scale bytes from end to end, the ends, 1.0 and 2^105's neighbours among them."""
    some = [254, 0, 127, 232, 1, 253, 233, 18, 126, 128, 64, 190, 105, 149, 20, 240]
    if n <= len(some):
        return torch.tensor(some[:n], dtype=torch.uint8, device="cuda")
    return (torch.arange(n, device="cuda") * 254 // (n - 1)).to(torch.uint8)


def as_bf16(v):
    """The nearest bf16 of doubles that are exact in fp32, or out of its range."""
    return v.float().to(torch.bfloat16)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("xc,wc", [(ONE, ONE), (TOP, TINY), (TINY, TOP), (TINY, TINY)])
def test_one_product_under_every_pair_of_scales(n, xc, wc):
    """One product per sum, a number of at most six bits: exact in bf16 where it is in its range,
    infinite above; zeros beside scales as large as they come stay zeros."""
    R, C = 255, 64
    x = torch.zeros(n, C, dtype=torch.uint8, device="cuda")
    w = torch.zeros(R, C, dtype=torch.uint8, device="cuda")
    x[:, 5], w[:, 5] = xc, wc
    xs, ws = (torch.full((r, C // 32), 254, dtype=torch.uint8, device="cuda") for r in (n, R))
    xs[:, 0] = token_bytes(n)
    ws[:, 0] = torch.arange(R, device="cuda")
    want = mx8_value(x.view(torch.float8_e4m3fn), xs) @ mx8_value(w.view(torch.float8_e4m3fn), ws).t()
    assert torch.equal(moe.linear(rows8(x, xs), rows8(w, ws)), as_bf16(want))


@pytest.mark.parametrize("n", ROWS)
def test_a_full_group_of_the_largest_codes(n):
    """32 products of 448 x 448, 49 x 2^17: the sum of the group passes 2^22 before its scales."""
    R, C = 255, 64
    x = torch.zeros(n, C, dtype=torch.uint8, device="cuda")
    w = torch.zeros(R, C, dtype=torch.uint8, device="cuda")
    x[:, 32:], w[:, 32:] = TOP, TOP
    xs, ws = (torch.zeros(r, C // 32, dtype=torch.uint8, device="cuda") for r in (n, R))
    xs[:, 1] = token_bytes(n)
    ws[:, 1] = torch.arange(R, device="cuda")
    want = mx8_value(x.view(torch.float8_e4m3fn), xs) @ mx8_value(w.view(torch.float8_e4m3fn), ws).t()
    assert torch.equal(moe.linear(rows8(x, xs), rows8(w, ws)), as_bf16(want))


@pytest.mark.parametrize("n", ROWS)
def test_groups_whose_scales_cancel(n):
    """Every group's two scales are far apart and their product is 1: the sums are those of the
    codes, small whole numbers, exact in fp32 in any order."""
    g = torch.Generator(device="cuda").manual_seed(n)
    R, C = 96, 512
    # whole numbers of -3 .. 3 as E4M3
    digit = torch.tensor([0xc4, 0xc0, 0xb8, 0x00, 0x38, 0x40, 0x44], dtype=torch.uint8, device="cuda")
    x = digit[torch.randint(7, (n, C), generator=g, device="cuda")]
    w = digit[torch.randint(7, (R, C), generator=g, device="cuda")]
    up = (torch.arange(C // 32, device="cuda") * 16 + 7).to(torch.uint8)     # 7 .. 247
    xs, ws = (254 - up).expand(n, -1).contiguous(), up.expand(R, -1).contiguous()
    want = x.view(torch.float8_e4m3fn).double() @ w.view(torch.float8_e4m3fn).double().t()
    assert torch.equal(moe.linear(rows8(x, xs), rows8(w, ws)), as_bf16(want))


@pytest.mark.parametrize("n", [1, 16, 40])
def test_gated_with_scales_far_apart(n):
    """The gated product shares the sums: the same rows under scales that cancel give the same h
    as under scales of 1."""
    g = torch.Generator(device="cuda").manual_seed(n)
    I, H = 96, 256
    digit = torch.tensor([0xb8, 0x00, 0x38], dtype=torch.uint8, device="cuda")   # -1, 0, 1
    x = digit[torch.randint(3, (n, H), generator=g, device="cuda")]
    w = digit[torch.randint(3, (2 * I, H), generator=g, device="cuda")]
    ones = [torch.full((r, H // 32), 127, dtype=torch.uint8, device="cuda") for r in (n, 2 * I)]
    up = torch.tensor([14, 240, 20, 234, 1, 253, 9, 245], dtype=torch.uint8, device="cuda")
    far = [(254 - up).expand(n, -1).contiguous(), up.expand(2 * I, -1).contiguous()]
    params = moe.make_params(act="swiglu", layout="packed")
    want = moe.gated_linear(rows8(x, ones[0]), rows8(w, ones[1]), params)
    assert torch.equal(moe.gated_linear(rows8(x, far[0]), rows8(w, far[1]), params), want)
    q = moe.gated_linear(rows8(x, far[0]), rows8(w, far[1]), params, mx8=True)
    p = moe.gated_linear(rows8(x, ones[0]), rows8(w, ones[1]), params, mx8=True)
    assert torch.equal(q.codes.view(torch.uint8), p.codes.view(torch.uint8))
    assert torch.equal(q.scales, p.scales)


@pytest.mark.parametrize("n", ROWS)
def test_a_scale_that_is_nan_beside_any_other(n):
    R, C = 255, 32
    x = torch.full((n, C), ONE, dtype=torch.uint8, device="cuda")
    w = torch.full((R, C), ONE, dtype=torch.uint8, device="cuda")
    xs, ws = token_bytes(n).view(n, 1), torch.arange(R, device="cuda").to(torch.uint8).view(R, 1)
    ws[77] = 255
    xs[n - 1] = 255
    got = moe.linear(rows8(x, xs), rows8(w, ws))
    bad = torch.zeros(n, R, dtype=torch.bool, device="cuda")
    bad[n - 1], bad[:, 77] = True, True
    assert torch.equal(torch.isnan(got), bad)


@pytest.mark.parametrize("n", ROWS)
@pytest.mark.parametrize("lo,hi", [(53, 190), (53, 191), (52, 190)])
def test_scales_around_the_border_of_the_two_orders(n, lo, hi):
    """Few rows take a shorter way where no scale lies outside bytes 53 to 190: all pairs within
    that range, and with the next byte at either end."""
    C = 96
    ends = torch.tensor([lo, hi, 127, 64], dtype=torch.uint8, device="cuda")
    xb = ends[torch.arange(n, device="cuda") % 4]
    wb = torch.arange(lo, hi + 1, device="cuda").to(torch.uint8)
    for code in (ONE, TINY, TOP):
        x = torch.zeros(n, C, dtype=torch.uint8, device="cuda")
        w = torch.zeros(len(wb), C, dtype=torch.uint8, device="cuda")
        x[:, 40], w[:, 40] = code, code
        xs, ws = xb[:, None].expand(-1, 3).contiguous(), wb[:, None].expand(-1, 3).contiguous()
        want = mx8_value(x.view(torch.float8_e4m3fn), xs) @ \
            mx8_value(w.view(torch.float8_e4m3fn), ws).t()
        assert torch.equal(moe.linear(rows8(x, xs), rows8(w, ws)), as_bf16(want)), code
