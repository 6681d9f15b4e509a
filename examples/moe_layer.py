"""A MoE layer trained and then served with 4-bit experts, and the dense block
(a shared expert) beside it.

    python examples/moe_layer.py train     # a few steps of gradient descent
    python examples/moe_layer.py decode    # the layer's experts in MXFP4, token by token
    python examples/moe_layer.py block     # norm, shared expert, residual: a few training
                                           # steps, then the same block in MXFP8

Training runs the experts as plain torch products on their contiguous slices
of the dispatched rows; the way there and back, and the gradients of both and
of the router's weights, are the library's calls:

    logits -> route_metadata -> dispatch -> experts -> combine_weighted -> out
    d_out -> combine_weighted_backward -> experts' backward -> dispatch_backward
          -> d_x; the weights' gradient -> route_backward -> d_logits

Serving quantises the experts once and calls forward_q4 for every step: three
kernels, no host synchronisation.

The block is three calls forward and three back:

    s, y = rms_norm(x, residual) -> h = gated_linear(y) -> out = linear(h) + s
    d_out -> linear_backward -> gated_linear_backward -> rms_norm_backward
          (+ d_out, through the residual) -> d_x
"""
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import mixture_experts_routing_warp_gb300 as moe  # noqa: E402

VALUES = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)   # E2M1 magnitudes


class Layer:
    """Router [E, H] fp32, experts w13 [E, 2I, H] (packed gate, up) and w2 [E, H, I]."""

    def __init__(self, H, E, I, k, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)

        def weight(*shape):
            w = torch.randn(*shape, generator=g, device="cuda") * shape[-1] ** -0.5
            return w.requires_grad_()

        self.H, self.E, self.I, self.k = H, E, I, k
        self.gate, self.w13, self.w2 = weight(E, H), weight(E, 2 * I, H), weight(E, H, I)

    def parameters(self):
        return [self.gate, self.w13, self.w2]

    def experts(self, rows, offs):
        """Each expert on its slice of the sorted rows; rows past the last stay zero."""
        parts = []
        for e in range(self.E):
            a = rows[offs[e]:offs[e + 1]] @ self.w13[e].t()
            gate, up = a.chunk(2, dim=1)
            parts.append((torch.nn.functional.silu(gate) * up) @ self.w2[e].t())
        parts.append(rows.new_zeros(rows.shape[0] - offs[-1], self.H))
        return torch.cat(parts)


def forward_backward(layer, x, d_out_of):
    """One pass and its gradients: out, and layer.*.grad and d_x for the
    gradient d_out_of(out)."""
    logits = x @ layer.gate.t()
    indx, vals, meta = moe.route_metadata(logits.detach(), layer.k)
    rows = moe.dispatch(x.detach(), meta, layer.k).requires_grad_()
    y = layer.experts(rows, meta["offs"].tolist())
    out = moe.combine_weighted(y.detach(), meta, vals)

    d_out = d_out_of(out)
    d_y, d_vals = moe.combine_weighted_backward(d_out, y.detach(), meta, vals)
    y.backward(d_y)                                      # experts' weights and rows
    d_x = moe.dispatch_backward(rows.grad, meta, layer.k)
    logits.backward(moe.route_backward(logits.detach(), indx, d_vals))  # the router
    return out, d_x


def train(H=256, E=8, I=256, k=2, n=512, steps=40, rate=0.15, seed=0):
    """The layer learns another layer's outputs; returns the losses."""
    teacher, layer = Layer(H, E, I, k, seed + 1), Layer(H, E, I, k, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    x = torch.randn(n, H, generator=g, device="cuda")
    target = forward_backward(teacher, x, torch.zeros_like)[0]
    losses = []
    for _ in range(steps):
        for p in layer.parameters():
            p.grad = None
        out, _ = forward_backward(layer, x, lambda o: 2.0 * (o - target) / n)
        losses.append(((out - target) ** 2).sum(dim=1).mean().item())
        with torch.no_grad():
            for p in layer.parameters():
                p -= rate * p.grad
    return losses


def quantise_mxfp4(w):
    """Codes [E, R, C/2] and scale bytes [E, R, C/32] of float weights [E, R, C]."""
    E, R, C = w.shape
    v = w.float().view(E, R, C // 32, 32)
    e = torch.floor(torch.log2(v.abs().amax(dim=3).clamp_min(2.0 ** -100))) - 2.0
    u = v / torch.exp2(e)[..., None]
    mids = torch.tensor([(a + b) / 2 for a, b in zip(VALUES, VALUES[1:])], device=w.device)
    code = (torch.bucketize(u.abs(), mids) + 8 * (u < 0)).view(E, R, C // 2, 2)
    codes = (code[..., 0] + 16 * code[..., 1]).to(torch.uint8)
    return codes.contiguous(), (e + 127.0).to(torch.uint8).contiguous()


def dequantise_mxfp4(codes, scales):
    """bf16 weights that the codes stand for (exact)."""
    table = torch.tensor(VALUES + tuple(-x for x in VALUES), device=codes.device)
    v = torch.stack((table[(codes & 15).long()], table[(codes >> 4).long()]), dim=-1).flatten(2)
    s = torch.exp2(scales.float() - 127.0).repeat_interleave(32, dim=2)
    return (v * s).to(torch.bfloat16)


def decode(H=2880, E=32, I=2880, k=4, tokens=8, seed=0):
    """`tokens` single-token steps with 4-bit experts, and the bf16 layer on
    the same (dequantised) weights; returns both outputs."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    q13, q2 = [], []
    for e in range(E):   # one expert at a time: the float weights need not fit together
        q13.append(quantise_mxfp4(torch.randn(1, 2 * I, H, generator=g, device="cuda") * 0.02))
        q2.append(quantise_mxfp4(torch.randn(1, H, I, generator=g, device="cuda") * 0.02))
    w13 = moe.Q4Weight(*(torch.cat(t) for t in zip(*q13)), "mxfp4")
    w2 = moe.Q4Weight(*(torch.cat(t) for t in zip(*q2)), "mxfp4")
    params = moe.make_params("softmax_topk", "swiglu_oai", "interleaved")
    ws = moe.workspace_q4(1, E, k, H, I)
    x = torch.randn(tokens, H, generator=g, device="cuda").to(torch.bfloat16)
    logits = torch.randn(tokens, E, generator=g, device="cuda")
    out = torch.empty_like(x)
    for t in range(tokens):
        moe.forward_q4(x[t:t + 1], logits[t:t + 1], w13, w2, k, params, ws, out=out[t:t + 1])

    full13 = dequantise_mxfp4(w13.codes, w13.scales)
    full2 = dequantise_mxfp4(w2.codes, w2.scales)
    want = moe.forward(x, logits, full13, full2, k, params, moe.workspace(tokens, E, k, H, I))
    return out, want


class Block:
    """norm [H], w13 [2I, H] (packed gate, up) and w2 [H, I], bf16 with fp32 masters."""

    def __init__(self, H, I, seed=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.params = moe.make_params(act="swiglu", layout="packed")
        self.master = [torch.ones(H, device="cuda"),
                       torch.randn(2 * I, H, generator=g, device="cuda") * H ** -0.5,
                       torch.randn(H, I, generator=g, device="cuda") * I ** -0.5]
        self.cast()

    def cast(self):
        self.norm, self.w13, self.w2 = (m.to(torch.bfloat16) for m in self.master)

    def forward(self, x, residual):
        """out, and what the backward pass needs."""
        y, s = moe.rms_norm(x, self.norm, residual=residual)
        h = moe.gated_linear(y, self.w13, self.params)
        return moe.linear(h, self.w2, residual=s), (y, s, h)

    def backward(self, d_out, kept):
        """(d_x, which is the residual's gradient too, and those of the weights)."""
        y, s, h = kept
        d_h, d_w2, _ = moe.linear_backward(d_out, h, self.w2)
        d_y, d_w13 = moe.gated_linear_backward(d_h, y, self.w13, self.params)
        d_x, d_norm = moe.rms_norm_backward(d_y, s, self.norm, d_sum=d_out)
        return d_x, (d_norm, d_w13, d_w2)


def quantise_mxfp8(w):
    """Mx8 rows of float weights [R, C]: E4M3 codes, the least scale of each 32
    under which none exceeds 448."""
    v = w.float().view(w.shape[0], -1, 32)
    e = torch.ceil(torch.log2(v.abs().amax(dim=2).clamp_min(2.0 ** -100) / 448.0))
    codes = (v / torch.exp2(e)[..., None]).view_as(w).to(torch.float8_e4m3fn)
    return moe.Mx8(codes, (e + 127.0).to(torch.uint8))


def serve_mxfp8(block, x, residual):
    """The block with 8 bits between its products: the norm and the gated
    product write them, the next product reads them."""
    y, s = moe.rms_norm(x, block.norm, residual=residual, mx8=True)
    h = moe.gated_linear(y, quantise_mxfp8(block.w13), block.params, mx8=True)
    return moe.linear(h, quantise_mxfp8(block.w2), residual=s)


def train_block(H=512, I=1408, n=1024, steps=20, rate=0.5, seed=0):
    """A block learns another's outputs; returns it, its losses and its inputs."""
    teacher, block = Block(H, I, seed + 1), Block(H, I, seed)
    g = torch.Generator(device="cuda").manual_seed(seed + 2)
    x, residual = (torch.randn(n, H, generator=g, device="cuda").to(torch.bfloat16)
                   for _ in range(2))
    target = teacher.forward(x, residual)[0]
    losses = []
    for _ in range(steps):
        out, kept = block.forward(x, residual)
        off = out.float() - target.float()
        losses.append((off ** 2).mean().item())
        _, grads = block.backward((off * (2.0 / n)).to(torch.bfloat16), kept)
        for m, d in zip(block.master, grads):
            m -= rate * d.float()
        block.cast()
    return block, losses, x, residual


if __name__ == "__main__":
    what = sys.argv[1] if len(sys.argv) > 1 else "train"
    if what == "train":
        for i, loss in enumerate(train()):
            print(f"step {i:2d}  loss {loss:.5f}")
    elif what == "block":
        block, losses, x, residual = train_block()
        for i, loss in enumerate(losses):
            print(f"step {i:2d}  loss {loss:.5f}")
        a, b = serve_mxfp8(block, x, residual), block.forward(x, residual)[0]
        err = (a.float() - b.float()).norm() / b.float().norm()
        print(f"in 8 bits: relative distance to the bf16 block {err:.5f}")
    else:
        a, b = decode()
        err = (a.float() - b.float()).norm() / b.float().norm()
        print(f"{a.shape[0]} tokens, relative distance to the bf16 layer {err:.5f}")
