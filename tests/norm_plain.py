"""Norms of heads' rows with the position rotation in 64 bits, for the tests, with the error bounds
that follow from the formats (roundings as in paged_plain)."""

import torch

from paged_plain import BF16, F32, turn64


def unit64(x, eps):
    """x [..., d] over the root of its mean square, and one over that root."""
    r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
    return x * r, r


def forward64(x, w, eps, angle=None, rot=0, interleaved=False):
    """The normed and turned rows, and what fp32 arithmetic may add before the last rounding."""
    d = x.shape[-1]
    y = unit64(x, eps)[0] * w
    # d squares summed, rsqrt (2 steps), two products
    slack = (d / 2 + 6) * F32 * y.abs()
    if angle is None:
        return y, slack
    out, more = turn64(y, angle, rot, interleaved)
    spread, _ = turn64(slack, torch.zeros_like(angle), rot, interleaved)
    # a pair's slack reaches both of its values
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    both = spread[..., a] + spread[..., b]
    spread[..., a] = spread[..., b] = both
    return out, more + spread


def backward64(x, w, eps, dy, angle=None, rot=0, interleaved=False):
    """dx and dw (summed over all rows) from dy, and their largest errors."""
    d = x.shape[-1]
    g, slack = (dy, torch.zeros_like(dy)) if angle is None else turn64(dy, -angle, rot, interleaved)
    u, r = unit64(x, eps)
    gw = g * w
    mean = (gw * u).mean(-1, keepdim=True)
    dx = r * (gw - u * mean)
    step = (d + 12) * F32
    mean_tol = ((slack * w.abs() + step * gw.abs()) * u.abs()).mean(-1, keepdim=True)
    dx_tol = r * (slack * w.abs() + step * (gw.abs() + (u * mean).abs()) + u.abs() * mean_tol) + \
        BF16 * dx.abs() * (1 + 2.0 ** -6) + 1e-30
    rows = x.numel() // d
    dims = tuple(range(x.dim() - 1))
    dw = (g * u).sum(dims)
    # rows products summed in fp32, in any order
    dw_tol = ((slack + (step + rows * F32) * g.abs()) * u.abs()).sum(dims) + 1e-30
    return dx, dw, dx_tol, dw_tol
