"""Attention with shaped scores in 64 bits, for the tests: scores and weights of a head whole, and
the error bounds that follow from the formats (roundings as in paged_plain)."""

import math

import torch

from paged_plain import BF16, F32

TANH = 2.0 ** -21  # of the capped score: the tanh (2e-7 of 1), ex2 and rcp within it


def spans_of(Nq, Nkv, causal=False, q_offset=0, window=0, first=None, end=None):
    """[Nq, Nkv] truth values: which keys each row sees."""
    pos = torch.arange(Nq)[:, None] + q_offset
    key = torch.arange(Nkv)[None, :]
    see = torch.ones(Nq, Nkv, dtype=torch.bool)
    if causal:
        see &= key <= pos
    if window:
        see &= key > pos - window
    if first is not None:
        see &= key >= first[:, None]
    if end is not None:
        see &= key < end[:, None]
    return see


class Head:
    """One query head in 64 bits: q [n, d], k and v [m, d], see [n, m]; forward and, with do,
    backward, each with the largest error that the kernels' roundings allow."""

    def __init__(self, q, k, v, see, scale, softcap=0.0, slope=0.0, q_offset=0, do=None):
        n, d = q.shape
        m = k.shape[0]
        raw = q @ k.T * scale
        size = q.abs() @ k.abs().T * scale
        y = torch.tanh(raw / softcap) if softcap else None
        x = softcap * y if softcap else raw
        g = 1 - y * y if softcap else torch.ones_like(raw)
        dist = (torch.arange(n)[:, None] + q_offset - torch.arange(m)[None, :]).abs().double()
        x = x - slope * dist
        live = see.any(1)
        x = x.masked_fill(~see, -math.inf)
        self.lse = torch.logsumexp(x, 1)
        p = torch.exp(x - self.lse.masked_fill(~live, 0.0)[:, None])
        self.o = p @ v
        self.live = live
        # Scores: d products summed in fp32, the tanh, the distance term and its product, the
        # exponent's sums (with lse) and ex2 (2^-22).
        big = torch.where(see, size + abs(slope) * dist, 0.0).amax(1) + self.lse.abs().masked_fill(
            ~live, 0.0)
        self.delta = (d + 8) * F32 * big + 2.0 ** -20 + TANH * softcap
        a = p @ v.abs()
        # P: rounded once to bf16; O: once.  (m sums in fp32.)
        self.o_tol = BF16 * self.o.abs() * (1 + 2.0 ** -6) + \
            (BF16 + 2 * self.delta[:, None] + m * F32) * a + 1e-30
        self.lse_tol = 2 * self.delta + 2 * F32 * self.lse.abs().masked_fill(~live, 0.0) + m * F32
        if do is None:
            return
        self.dv = p.T @ do
        dp = do @ v.T
        D = (p * dp).sum(1, keepdim=True)
        ds = p * g * (dp - D)
        self.dq, self.dk = ds @ k * scale, ds.T @ q * scale
        # P from the saved lse: delta twice.  D: of O as the forward left it, or of P and dP.
        two = 2 * self.delta[:, None] + F32 * m
        dp_tol = d * F32 * (do.abs() @ v.abs().T)
        D_tol = (do.abs() * self.o_tol).sum(1, keepdim=True) + d * F32 * (do.abs() * a).sum(
            1, keepdim=True) + (p * (dp_tol + two * dp.abs())).sum(1, keepdim=True)
        # a cap's 1 - tanh^2: twice the tanh's error; dS: rounded to bf16
        ds_tol = p * ((g * (1 + 2 * two)) * (dp_tol + D_tol) + 4 * TANH * (dp - D).abs()) + \
            (two + BF16) * ds.abs()
        # a row of one key has dS = 0 in the kernels, as here but for this sum's own rounding
        self.dv_tol = (p * (BF16 + two + n * F32)).T @ do.abs()
        self.dq_tol = ds_tol @ k.abs() * scale + BF16 * self.dq.abs() * (1 + 2.0 ** -6) + 1e-30
        self.dk_tol = ds_tol.T @ q.abs() * scale + n * F32 * (ds.abs().T @ q.abs()) * scale


def whole(q, k, v, see, scale, softcap=0.0, slopes=None, q_offset=0, do=None):
    """The same of [B, H, N, d] tensors (see: a list of B): a dict of values and of bounds."""
    B, Hq, n, d = q.shape
    Hkv, m = k.shape[1:3]
    val = {"o": torch.zeros(q.shape), "lse": torch.zeros(q.shape[:3])}
    if do is not None:
        val.update(dq=torch.zeros(q.shape), dk=torch.zeros(k.shape), dv=torch.zeros(k.shape))
    val = {a: x.double() for a, x in val.items()}
    tol = {a: torch.zeros_like(x) for a, x in val.items()}
    for b in range(B):
        for h in range(Hq):
            hk = h // (Hq // Hkv)
            x = Head(q[b, h].double(), k[b, hk].double(), v[b, hk].double(), see[b], scale, softcap,
                     0.0 if slopes is None else float(slopes[h]), q_offset,
                     None if do is None else do[b, h].double())
            val["o"][b, h], tol["o"][b, h] = x.o, x.o_tol
            val["lse"][b, h], tol["lse"][b, h] = x.lse, x.lse_tol
            if do is not None:
                val["dq"][b, h], tol["dq"][b, h] = x.dq, x.dq_tol
                for a in ("dk", "dv"):  # a shared head's are sums over its query heads
                    val[a][b, hk] += getattr(x, a)
                    tol[a][b, hk] += getattr(x, a + "_tol")
    for a in ("dk", "dv"):
        if do is not None:
            tol[a] += BF16 * val[a].abs() * (1 + 2.0 ** -6) + 1e-30
    return val, tol


def off_by(got, val, tol):
    """The largest share of its bound that an error takes; infinite where a value that has none
    (a row that sees no key) is not that value."""
    got = got.double().cpu()
    odd = ~torch.isfinite(val)
    if not torch.equal(torch.where(odd, got, 0.0), torch.where(odd, val, 0.0)):
        return math.inf
    err = torch.where(odd, 0.0, got - val).abs()
    if torch.isnan(err).any():
        return math.inf
    return (err / torch.where(odd, 1.0, tol)).max().item()
