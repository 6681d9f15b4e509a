"""The dense blocks' formulas in 64 bits, and how far a kernel may be off.

Bounds. A sum of K products in fp32 is off by at most K * 2^-23 times the sum
of the products' magnitudes (2^-24 for each rounding to nearest; 2^-23 covers
an addition that cuts bits off, as a tensor core's may), a result by half a
step of its type more. An intermediate that is rounded to 16 bits brings
eps / 2 of each product it enters. The sigmoid and the other functions are
good to 2^-19 of their value.
"""
import math

import torch

DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
FN = 2.0 ** -19


def half_step(dtype):
    return torch.finfo(dtype).eps / 2


def tiny(dtype):
    """Half the distance of the subnormal values."""
    return torch.finfo(dtype).smallest_normal * torch.finfo(dtype).eps / 2


def check(got, want, slack, what=""):
    """|got - want| <= slack + half a step of got's type, element by element."""
    assert got.shape == want.shape, (got.shape, want.shape)
    g = got.double()
    assert torch.equal(torch.isfinite(g), torch.isfinite(want)), what
    # half a step of the rounded value: relative to the value with its slack
    bound = slack + (want.abs() + slack) * half_step(got.dtype) + tiny(got.dtype)
    off = (g - want).abs() - bound
    off = torch.where(torch.isfinite(want), off, torch.full_like(off, -1.0))
    assert off.numel() == 0 or off.max() <= 0, \
        f"{what}: {off.max().item():.3g} over the bound at {off.argmax().item()}"


def randn(g, *shape, dtype=torch.bfloat16, scale=1.0):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def product(x, w):
    """(x w^T, what fp32 sums of it may be off)."""
    x, w = x.double(), w.double()
    return x @ w.t(), (x.abs() @ w.abs().t()) * (x.shape[1] * 2.0 ** -23)


ACTS = {
    "none": (lambda v: v, lambda v: torch.ones_like(v)),
    "silu": (lambda v: v * torch.sigmoid(v),
             lambda v: torch.sigmoid(v) * (1 + v * (1 - torch.sigmoid(v)))),
    "gelu": (lambda v: 0.5 * v * (1 + torch.erf(v / math.sqrt(2))),
             lambda v: 0.5 * (1 + torch.erf(v / math.sqrt(2))) +
             v * torch.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)),
    "relu2": (lambda v: torch.relu(v) ** 2, lambda v: 2 * torch.relu(v)),
}


def act_slack(a, da, act):
    """How far act(a) may be off for an argument off by da: the slope is at most
    1.13 for silu and gelu, 2 |a + da| for relu2."""
    slope = {"none": 1.0, "silu": 1.13, "gelu": 1.13}.get(act, 2 * (a.abs() + da))
    return slope * da + (0 if act == "none" else a.abs() * FN * (a.abs() + 1 if act == "relu2" else 1))


def slope_slack(a, da, act):
    """The same for act'(a): the second derivative is at most 1 (0.5 for silu,
    0.8 for gelu), 2 for relu2."""
    if act == "none":
        return torch.zeros_like(a)
    return 2 * da + FN * (1 + a.abs())


def halves(a, layout):
    if layout == "packed":
        return a[:, :a.shape[1] // 2], a[:, a.shape[1] // 2:]
    return a[:, 0::2], a[:, 1::2]


def joined(g, u, layout):
    return torch.cat((g, u), 1) if layout == "packed" else torch.stack((g, u), 2).flatten(1)


class Gate:
    """The gated activation with its parameters resolved."""

    def __init__(self, act="swiglu", alpha=None, beta=None, limit=None):
        oai = act == "swiglu_oai"
        self.alpha = (1.702 if alpha is None else alpha) if oai else 1.0
        self.beta = (1.0 if beta is None else beta) if oai else 0.0
        self.limit = limit if limit is not None else (7.0 if oai else math.inf)

    def clamped(self, g, u):
        return g.clamp(max=self.limit), u.clamp(-self.limit, self.limit)

    def forward(self, g, u, dg, du):
        """h, and what it may be off for arguments off by dg, du."""
        gc, uc = self.clamped(g, u)
        s = torch.sigmoid(self.alpha * gc)
        h = gc * s * (uc + self.beta)
        # d(g s(alpha g))/dg <= 1.1; |g s| <= |g|
        slack = 1.1 * dg * ((uc + self.beta).abs() + du) + (gc.abs() + dg) * s.clamp_min(2 ** -20) * du
        return h, slack + h.abs() * FN + 2 ** -24 * gc.abs() * (uc.abs() + abs(self.beta))

    def backward(self, g, u, d, dg, du):
        """(d_g, d_u), and what each may be off, before any rounding."""
        gc, uc = self.clamped(g, u)
        s = torch.sigmoid(self.alpha * gc)
        up = uc + self.beta
        slope = s * (1 + self.alpha * gc * (1 - s))
        d_g, d_u = d * up * slope, d * gc * s
        zero = torch.zeros_like(d)
        near_g, near_u = (g - self.limit).abs() <= dg, (u.abs() - self.limit).abs() <= du
        d_g = torch.where(g <= self.limit, d_g, zero)
        d_u = torch.where(u.abs() <= self.limit, d_u, zero)
        # slope' is at most alpha (|slope'| of silu is at most 0.5)
        fn = FN * (1 + self.alpha * gc.abs())
        e_g = d.abs() * (du * (1 + fn) * 1.2 + (up.abs() + du) * (max(self.alpha, 1) * dg + fn))
        e_u = d.abs() * (1.1 * dg + FN * (gc.abs() + dg))
        # at the limit either side may be taken
        e_g = torch.where(near_g, e_g + (d * up * slope).abs(), e_g)
        e_u = torch.where(near_u, e_u + (d * gc * s).abs(), e_u)
        return d_g, d_u, e_g, e_u


# ------------------------------------------------------------------ MXFP8 --
def mx8_scale(v):
    """[rows, C/32] scale bytes of rows v (double): the least power of two under
    which no value exceeds 448; 255 for a group that is not finite."""
    group = v.unflatten(1, (-1, 32))
    m, e = torch.frexp(group.abs().amax(dim=2).nan_to_num(0.0, 0.0, 0.0))
    e = torch.where(m <= 0.875, e - 9, e - 8)
    e = torch.where(m == 0, torch.full_like(e, -127), e).clamp(-127, 127)
    bad = ~torch.isfinite(group).all(dim=2)
    return torch.where(bad, torch.full_like(e, 255), e + 127)


def mx8_value(codes, scales):
    """double rows that codes and scale bytes stand for."""
    s = torch.exp2(scales.double() - 127.0)
    s = torch.where(scales == 255, torch.full_like(s, math.nan), s)
    return codes.float().double() * s.repeat_interleave(32, dim=1)


def mx8_rows(g, rows, cols, scale=1.0):
    """Random MXFP8 rows (codes, scale bytes)."""
    v = torch.randn(rows, cols, generator=g, device="cuda").double() * scale
    b = mx8_scale(v)
    u = v * torch.exp2(127.0 - b.double()).repeat_interleave(32, dim=1)
    return u.float().to(torch.float8_e4m3fn), b.to(torch.uint8)


def check_mx8(codes, scales, want, slack, what=""):
    """Quantised rows against the values before their rounding (double). The
    scale may be the next one where the group's largest value lies within its
    slack of the border; a code is off by half a step of E4M3 (2^-4 of its
    value, 2^-10 of the scale for its subnormals)."""
    top = want.unflatten(1, (-1, 32)).abs().amax(dim=2)
    s = slack.expand_as(want).unflatten(1, (-1, 32)).amax(dim=2)
    low = mx8_scale((top - s).clamp_min(0).repeat_interleave(32, dim=1))
    high = mx8_scale((top + s).repeat_interleave(32, dim=1))
    b = scales.long()
    assert ((b >= low) & (b <= high)).all(), f"{what}: scales"
    got = mx8_value(codes, scales)
    unit = torch.exp2(b.double() - 127.0).repeat_interleave(32, dim=1)
    bound = slack + (want.abs() + slack) * 2.0 ** -4 + unit * 2.0 ** -10
    assert ((got - want).abs() <= bound).all(), f"{what}: values"
