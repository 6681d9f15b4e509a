"""MXFP4 rows whose group scales are too far apart for one fp16 reference."""
import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from test_q4_gpu import BF16, check, decode64, product64, random_q4, tokens

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n", [3, 12])
def test_infinity_beside_far_scales(n):
    """Group scales of a row too far apart for one reference, in some rows of
    a tile: an infinite activation still gives infinities in every row."""
    C, R = 416, 50
    w, x = random_q4((R, C), "mxfp4", 170), tokens(n, C, BF16, 171)
    g = torch.Generator(device="cuda").manual_seed(172)
    far = torch.randint(77, 178, w.scales.shape, generator=g, device="cuda", dtype=torch.uint8)
    w.scales[::3] = far[::3]
    w.codes[:, 20] = 0x19          # columns 40 and 41: -0.5 and 0.5 everywhere
    W = decode64(w)
    x[1, 40] = float("inf")
    out = moe.linear_q4(x, w)
    assert torch.equal(out[1], torch.full_like(out[1], float("-inf")))
    keep = [t for t in range(n) if t != 1]
    check(out[keep], *product64(x[keep].double(), W))


@pytest.mark.parametrize("n", [1, 12])
@pytest.mark.parametrize("zero_scale", [25, 85, 0])
def test_groups_of_zeros(n, zero_scale):
    """A quantiser gives a group of zeros a scale far below the others': first
    in a row, in the middle, whole slabs of them, whole rows."""
    C, R = 1024, 48
    w, x = random_q4((R, C), "mxfp4", 180), tokens(n, C, BF16, 181)
    codes, scales = w.codes.view(R, C // 32, 16), w.scales
    for r, groups in ((0, [0]), (1, [0, 1, 2, 3]), (2, [5]), (3, range(8, 16)), (4, range(32)),
                      (5, range(31)), (21, [31]), (40, range(0, 32, 2))):
        for j in groups:
            codes[r, j], scales[r, j] = 0x80 if r % 2 else 0, zero_scale
    check(moe.linear_q4(x, w), *product64(x.double(), decode64(w)))


@pytest.mark.parametrize("n", [1, 12])
def test_scales_that_climb_and_fall(n):
    """Rows whose scales rise or fall along the row by more than one
    reference holds, with activations on the small groups alone too."""
    C, R = 2048, 20
    w, x = random_q4((R, C), "mxfp4", 190), tokens(n, C, BF16, 191)
    up = torch.linspace(70, 180, C // 32, device="cuda").to(torch.uint8)
    w.scales[::2], w.scales[1::2] = up, up.flip(0)
    w.scales[7] = 200
    W = decode64(w)
    check(moe.linear_q4(x, w), *product64(x.double(), W))
    for lo in (0, 256, C - 256):   # the columns of the largest scales left out for some rows
        only = torch.zeros_like(x)
        only[:, lo:lo + 256] = x[:, lo:lo + 256]
        ref, err = product64(x[:, lo:lo + 256].double(), W[:, lo:lo + 256])
        check(moe.linear_q4(only, w), ref, err)
