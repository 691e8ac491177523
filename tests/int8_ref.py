"""The int8 operators and the norms in 64 bits, from their definitions (CPU)."""

import math

import torch

HALF = 2.0 ** -8    # half a bf16 step, relative to the value
TINY = 2.0 ** -134  # half the smallest bf16 number


def quantize(x):
    """(codes int8, scale float32) of the rows of x (bf16).  The quotients are formed in 64 bits and rounded to 32:
    that is the correctly rounded 32-bit quotient (53 >= 2 * 24 + 2 bits)."""
    x = x.double()
    amax = x.abs().amax(1, keepdim=True)
    fine = torch.isfinite(x).all(1, keepdim=True)
    s = (amax / 127).float()
    s = torch.where(amax == 0, 1.0, s)
    q = (x / s.double()).float().double()
    codes = torch.where(fine, torch.round(q), 0.0)
    assert float(codes.abs().max() if codes.numel() else 0) <= 127
    return codes.to(torch.int8), torch.where(fine, s, math.nan)[:, 0]


def product(codes, scale, w, ws):
    """s_row * s_col * sum, in 64 bits (the sum is exact: below 2^31)."""
    acc = codes.double() @ w.double().t()
    return acc * scale.double()[:, None] * ws.double()


def product_bound(ref):
    """|gpu - ref|: the sum rounded to fp32, two products and the power of two (2^-24 each), then bf16."""
    return ref.abs() * (HALF + 4 * 2.0 ** -24) + TINY


def norm(x, weight, offset, eps):
    x = x.double()
    n = x / torch.sqrt((x * x).mean(1, keepdim=True) + eps)
    return n if weight is None else n * (offset + weight.double())


def norm_rel(k):
    """Relative error of the fp32 norm before its rounding.  The sum of squares: a thread adds up to 8 squares of each
    of its at most 16 pieces, six steps join a wave, up to 16 add the waves; each square is rounded with its sum (or,
    scaled, exactly before).  All terms are positive, so the sum is off by (144 + 22) * 2^-24, its root by half of
    that, the mean, eps, the reciprocal root and its square's rounding by 4 steps, the products by 3."""
    return (83 + 7) * 2.0 ** -24


def norm_bound(ref, k):
    return ref.abs() * (HALF + norm_rel(k)) + TINY


def residual(residual, y, post, gate, scale, offset, eps):
    """(h, its bound).  post: None, True or weights; gate: None or [gates, k]."""
    t = y.double() if post is None else norm(y, None if post is True else post, offset, eps)
    m = y.shape[0]
    if gate is not None:
        gate = gate.reshape(-1, y.shape[1]).double()
        t = t * gate.repeat_interleave(m // gate.shape[0], 0)
    t = scale * t
    h = residual.double() + t
    # what is added is off by norm_rel and two products; the sum is rounded to fp32 and to bf16
    return h, h.abs() * (HALF + 2.0 ** -23) + t.abs() * (norm_rel(y.shape[1]) + 3 * 2.0 ** -24) + TINY
