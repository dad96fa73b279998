"""Reference forms of the block operators in 64 bits, and how far fp32 arithmetic with one rounding to
the result's type may be from them. Used by the GPU tests; their own tests are in test_block_host.py.

U is half a step of fp32 relative to the value (2^-24). A sum of n products that are exact in fp32,
in any order, is off by (n - 1) U times the sum of the products' sizes at most (first order; 1.01
covers the rest); each further operation adds U of its result. A rounding to fp16 is off by 2^-11 of
the value, or 2^-25 where the value is subnormal.
"""
import math

import torch

U = 2.0 ** -24
SLOPE = 1.13          # the activations' largest derivative (gelu's at sqrt 2: 1.129)
EXPONENTS = {None: 0.0, "none": 0.0, "relu": 0.0, "silu": 1.0, "gelu": 0.0, "gelu_tanh": 1.0}


def act(x, name):
    """The activation in 64 bits."""
    if name in (None, "none"):
        return x
    if name == "relu":
        return x.clamp(min=0)
    if name == "silu":
        return x * torch.special.expit(x)
    if name == "gelu":
        return x * torch.special.ndtr(x)
    return x * torch.special.expit(2.0 * math.sqrt(2.0 / math.pi) * (x + 0.044715 * x ** 3))


def act_slack(x, name):
    """How far the kernels' activation of an exact x may be. The logistic forms: exp's argument t has
    three roundings or fewer before its product with log2 e, which moves exp by 4 |t| U relative, and
    v_exp, the sum, v_rcp and the last product are within 8 U together. erfc: 8 U (its argument's
    rounding moves it by x^2 U relative at most, counted for x^2 <= 60, past which fp16 has 0)."""
    y = act(x, name).abs()
    if name in (None, "none", "relu"):
        return torch.zeros_like(y)
    if name == "gelu":
        return y * (8.0 + x.square().clamp(max=60.0)) * U
    t = x.abs() if name == "silu" else 1.6 * x.abs() * (1.0 + 0.045 * x.square())
    return y * (8.0 + 4.0 * t) * U


def half_rounding(y):
    return torch.maximum(2.0 ** -11 * y.abs(), torch.full_like(y, 2.0 ** -25))


def product(x, w, bias):
    """(x W^T + bias, its fp32 slack): x, w (the pruned matrix) in 64 bits."""
    y = x @ w.t()
    size = x.abs() @ w.abs().t()
    kept = int((w != 0).sum(1).max()) if w.numel() else 0
    slack = 1.01 * (kept + 1) * U * size
    if bias is not None:
        y = y + bias
        slack = slack + U * (y.abs() + slack)
    return y, slack


def linear(x, w, bias, name, scale, residual):
    """(the result in 64 bits, the largest distance of a right fp16 result)."""
    s, slack = product(x, w, bias)
    y = scale * act(s, name)
    slack = abs(scale) * (SLOPE * slack + act_slack(s, name))
    if residual is not None:
        y = y + residual
    slack = slack + 2.0 * U * (y.abs() + slack)
    return y, slack + half_rounding(y)


def gated(x, wg, wu, bg, bu, name):
    g, gs = product(x, wg, bg)
    u, us = product(x, wu, bu)
    a = act(g, name)
    sa = SLOPE * gs + act_slack(g, name)
    y = a * u
    slack = sa * u.abs() + a.abs() * us + sa * us
    slack = slack + U * (y.abs() + slack)
    return y, slack + half_rounding(y)


def norm(x, weight, bias, kind, offset, eps, before=None):
    """(norm of x in 64 bits, its fp32 slack); before: the slack of x."""
    n = x.shape[-1]
    d = torch.zeros_like(x) if before is None else before
    if kind == "layer":
        mean = x.mean(-1, keepdim=True)
        # the mean: a sum of n, a division; then a subtraction
        moved = (n + 1) * U * x.abs().mean(-1, keepdim=True) + d.mean(-1, keepdim=True)
        x = x - mean
        d = d + moved + U * x.abs()
    square = x.square().mean(-1, keepdim=True)
    # the sum of squares' relative slack: its n + 3 roundings, and twice the elements' own; rsqrt halves it
    off = (n + 4) * U + 2.0 * (x.abs() * d + d.square()).mean(-1, keepdim=True) / square.clamp(min=1e-300)
    r = 1.0 / torch.sqrt(square + eps)
    share = square / (square + eps).clamp(min=1e-300)
    y = x * r
    slack = d * r + y.abs() * (0.5 * off * share + 4.0 * U) + d * r * off
    if weight is not None:
        f = offset + weight
        y, slack = y * f, slack * f.abs() + 2.0 * U * (y * f).abs()
    if bias is not None:
        y = y + bias
        slack = slack + U * y.abs()
    return y, slack


def block_norm(x, branch, weight, bias, post, gate, scale, kind, offset, eps):
    """((y, slack), (h, slack)), without the last roundings."""
    b, d = branch, torch.zeros_like(branch)
    if post is not None:
        b, d = norm(branch, post, None, kind, offset, eps)
    if gate is not None:
        b, d = b * gate, d * gate.abs() + U * (b * gate).abs()
    h = x + scale * b
    d = abs(scale) * d + U * (h.abs() + (scale * b).abs())
    return norm(h, weight, bias, kind, offset, eps, d), (h, d)


def scores(z):
    """log p of rows of scaled logits in 64 bits (NaN where a row has NaN or +infinity, -infinity where
    it has nothing else), and their entropy."""
    bad = z.isnan().any(-1) | (z == math.inf).any(-1)
    none = ~bad & (z == -math.inf).all(-1)
    top = z.max(-1, keepdim=True)
    d = z - top.values                    # before the logarithm, whose digits a large z would swallow,
    e = d.exp().scatter(-1, top.indices, 0.0)      # and 1 apart from the other terms
    lp = d - torch.log1p(e.sum(-1, keepdim=True))
    lp = torch.where(none[:, None], torch.full_like(lp, -math.inf), lp)
    p = lp.exp()
    entropy = -torch.where(p > 0, p * lp, torch.zeros_like(p)).sum(-1)
    nan = torch.full_like(entropy, math.nan)
    return torch.where(bad[:, None], nan[:, None], lp), torch.where(bad, nan, entropy)


def best(x, top):
    """The `top` best of each row by (value, lower index), -1 where there is no more above -infinity."""
    order = torch.sort(-x.double(), dim=-1, stable=True).indices[:, :top]
    return torch.where(x.gather(1, order) > -math.inf, order, -1)
