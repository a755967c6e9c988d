"""A server's steps for the tests: three sequences that grow by prompts in chunks and by single
tokens, and the largest error that attention over what the pages hold may have."""

import math

import torch

from paged_plain import BF16, E4M3, F16, F32, angles64, attention64, turn64

D, HQ, HKV, PAGE = 128, 8, 2, 16
TOTAL = (150, 97, 40)
STEPS = [[70, 0, 40], [1, 90, 0], [64, 1, 0]] + [[1, 1, 0]] * 5 + [[10, 1, 0]]
INV_FREQ = (10000.0 ** (-torch.arange(D // 2, dtype=torch.float64) * 2 / D)).float()


def inputs(seed=5):
    """q, k and v of every sequence, [n, heads, D] bf16."""
    g = torch.Generator().manual_seed(seed)
    return [tuple(torch.randn(n, h, D, generator=g).to(torch.bfloat16) for h in (HQ, HKV, HKV))
            for n in TOTAL]


def turned(x, first):
    """x [n, heads, D] at places first, first + 1, ... in 64 bits, and the slack of fp32."""
    place = torch.arange(first, first + x.shape[0])[None]
    angle = angles64(place, INV_FREQ, torch.zeros(D // 2))[:, None]
    return turn64(x.double(), angle, D, False)


def stored_bound(want, slack, descale, e4m3):
    """What one rounding to the cache's type may be off, of values / descale."""
    w = want.abs() / descale
    rounding = (E4M3 * w).clamp(min=2.0 ** -10) if e4m3 else BF16 * w
    return rounding * (1 + 2.0 ** -6) + slack / descale + 1e-30


def attention_bound(o, lse, a, size, m, v_max, e4m3):
    """Largest |error| of o and lse against 64-bit values over the very bits that are read: the
    scores' sums and exponentials (delta, twice), P's rounding, O's rounding; fp16 weights end
    2^-32 below the largest."""
    delta = (D + 8) * F32 * (size + lse.abs()) + 2.0 ** -20
    o_tol = BF16 * o.abs() * (1 + 2.0 ** -6) + \
        ((F16 if e4m3 else BF16) + 2 * delta[..., None]) * a
    if e4m3:
        o_tol = o_tol + m * 2.0 ** -32 * (1 + 2.0 ** -6) * v_max
    return o_tol + 1e-30, 2 * delta + 2 * F32 * lse.abs()


def exact(q, k, v):
    """The newest q [n, HQ, D] over k and v [m, HKV, D] in 64 bits, with attention64's sums."""
    return attention64(q, k, v, 1 / math.sqrt(D), True, k.shape[0] - q.shape[0])
