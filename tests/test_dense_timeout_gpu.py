"""A wait of the dense products' roles that runs out: the product gives up, says so in its
status word and leaves the device as usable as before."""
import os
import subprocess
import sys
import time

import pytest
import torch

import mixture_experts_routing_warp_gb300 as moe
from mixture_experts_routing_warp_gb300 import build as cuda_build

MS = 1_000_000
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
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
    for spoil in ({"x": None}, {"w": None}, {"y": None}, {"ns": 0},
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


@pytest.mark.gpu
def test_a_call_without_a_status_word_is_not_silent():
    """What a call without a status word records is found in the device's own, by every kind
    of call; one with a word of its own leaves that alone."""
    g = torch.Generator(device="cuda").manual_seed(1)
    x, w = (torch.randn(300, 256, generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
    y, st = torch.empty(300, 300, dtype=torch.bfloat16, device="cuda"), \
        torch.zeros(1, dtype=torch.int32, device="cuda")
    size = moe.linear_workspace_size(300, 300, 256)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda") if size else None
    assert moe.read_status() == 0
    assert starve(x, w, y, ws, None, 5 * MS) == 0
    assert moe.read_status() == TIMEOUT
    moe.linear(x, w)
    assert moe.read_status(reset=True) == TIMEOUT     # kept until it is reset
    assert moe.read_status() == 0
    assert starve(x, w, y, ws, st, 5 * MS) == 0
    assert moe.read_status() == 0 and st.item() == TIMEOUT
    # captured, on a stream of its own
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        assert starve(x, w, y, ws, None, 5 * MS) == 0
    assert moe.read_status() == 0
    graph.replay()
    assert moe.read_status(reset=True) == TIMEOUT
    assert torch.equal(moe.linear(x, w), moe.linear(x, w, status=st.zero_()))
    assert moe.read_status() == 0 and st.item() == 0


FIRST = """
import torch, mixture_experts_routing_warp_gb300 as moe
x = torch.ones(64, 256, dtype=torch.bfloat16, device="cuda")
out = torch.empty(64, 64, dtype=torch.bfloat16, device="cuda")
ws = torch.empty(max(1, moe.linear_workspace_size(64, 64, 256)), dtype=torch.uint8, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    moe.linear(x, x, out=out, ws=ws)
graph.replay()
torch.cuda.synchronize()
assert (out == 256).all() and moe.read_status() == 0
"""


@pytest.mark.gpu
def test_the_first_call_of_a_process_may_be_a_captured_one():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
