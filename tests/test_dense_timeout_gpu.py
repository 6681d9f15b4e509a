"""A wait of the dense products' roles that runs out: the product gives up, says so in its
status word and leaves the device as usable as before."""
import time

import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from mixture_experts_routing_warp_gb300 import build as cuda_build

MS = 1_000_000
TIMEOUT = 5                    # MOE_ERR_TIMEOUT


def starve(x, w, y, ws, status, ns, n=None, R=None, C=None, dtype=0):
    """The self-test on tensors, or on addresses (never read) with sizes."""
    at = lambda t: t.data_ptr() if isinstance(t, torch.Tensor) else t  # noqa: E731
    n, R, C = n if n is not None else x.shape[0], R or w.shape[0], C or x.shape[1]
    size = ws.numel() if isinstance(ws, torch.Tensor) else (0 if ws is None else 1 << 40)
    stream = torch.cuda.current_stream().cuda_stream if isinstance(x, torch.Tensor) else None
    return moe.lib().moe_selftest_linear_timeout(at(x), at(w), n, R, C, dtype, at(y), at(ws), size,
                                                 ns, at(status), stream)


def test_refusals():
    cuda_build.build()
    P = 1 << 20
    good = dict(x=P, w=P, y=P, ws=P, status=P, ns=MS, n=100, R=64, C=2880)
    for spoil in ({"x": None}, {"w": None}, {"y": None}, {"status": None}, {"ns": 0},
                  {"ns": 10 ** 9 + 1}, {"n": 0}, {"n": 16}, {"R": 1 << 20}, {"C": 60},
                  {"dtype": 2}):
        assert starve(**dict(good, **spoil)) == 1, spoil
    for spoil in ({"x": P + 8}, {"w": P + 8}, {"y": P + 1}, {"status": P + 2}):
        assert starve(**dict(good, **spoil)) == 6, spoil


# the last copy issued before a wait runs out (2 steps); the ring full (45); several
# tiles per pair of CTAs; a sum in parts
@pytest.mark.gpu
@pytest.mark.parametrize("n,R,C", [(256, 512, 128), (256, 512, 2880), (4096, 2880, 320),
                                   (200, 256, 8192)])
def test_a_wait_that_runs_out(n, R, C):
    g = torch.Generator(device="cuda").manual_seed(n)
    x = torch.randn(n, C, generator=g, device="cuda").to(torch.bfloat16)
    w = torch.randn(R, C, generator=g, device="cuda").to(torch.bfloat16)
    want = moe.linear(x, w)
    y = torch.empty_like(want)
    size = moe.linear_workspace_size(n, R, C)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    st = torch.zeros(1, dtype=torch.int32, device="cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        t = time.monotonic()
        assert starve(x, w, y, ws, st, 20 * MS) == 0
        torch.cuda.synchronize()
        # 20 ms at 3 cycles per ns, then 2 ms for each of at most 8 stages, at any clock
        assert time.monotonic() - t < 2.0
        assert st.item() == TIMEOUT
        st.zero_()
        assert torch.equal(moe.linear(x, w, status=st), want)   # right behind it
        assert st.item() == 0
