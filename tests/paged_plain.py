"""Rotary positions and paged attention in 64 bits, for the tests: plain loops
over sequences and heads, and the error bounds that follow from the formats.

A rounding is off by at most half a step, 2^-8 of the value for bf16, 2^-11 for
fp16, 2^-24 for fp32, 2^-4 for e4m3 (2^-10 absolute below its normal range).
"""

import math

import torch

BF16, F16, F32, E4M3 = 2.0 ** -8, 2.0 ** -11, 2.0 ** -24, 2.0 ** -4


def turn64(x, angle, rot, interleaved):
    """x [..., d] in 64 bits with its pairs turned by angle [..., rot / 2]."""
    y = x.clone()
    i = torch.arange(rot // 2)
    a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
    c, s = torch.cos(angle), torch.sin(angle)
    y[..., a] = x[..., a] * c - x[..., b] * s
    y[..., b] = x[..., a] * s + x[..., b] * c
    # what the fp32 arithmetic may add: the angle as a fraction of a turn (2^-25 of one from its
    # conversion to fp32, 2^-32 from the cut, times 2 pi), sine and cosine to two steps, and three
    # roundings of products and their sum; together under 2^-20 of the pair
    size = x.abs()
    slack = torch.zeros_like(x)
    slack[..., a] = slack[..., b] = 2.0 ** -20 * (size[..., a] + size[..., b])
    return y, slack


def angles64(positions, inv_freq, axis):
    """positions [axes, ...] int, axis [rot / 2] -> [..., rot / 2]."""
    p = positions.double()[axis.long()]
    return p.movedim(0, -1) * inv_freq.double()


def attention64(q, k, v, scale, causal, offset):
    """q [n, H, d], k and v [m, Hkv, d] (the m keys seen by anyone), 64 bits: o, lse, and per
    element sum_j w_j |v_j| and per row the largest scale * sum |q||k|."""
    n, H, d = q.shape
    m, Hkv = k.shape[:2]
    G = H // Hkv
    qq = q.view(n, Hkv, G, d)
    s = torch.einsum("nhgd,mhd->nhgm", qq, k) * scale
    size = torch.einsum("nhgd,mhd->nhgm", qq.abs(), k.abs()) * scale
    see = torch.arange(m)[None, :] <= (torch.arange(n)[:, None] + offset if causal else
                                       torch.full((n, 1), m))
    s = s.masked_fill(~see[:, None, None], -math.inf)
    size = size.masked_fill(~see[:, None, None], 0.0)
    if m == 0:
        z = torch.zeros(n, H, d, dtype=torch.float64)
        return z, torch.full((n, H), -math.inf, dtype=torch.float64), z, torch.zeros(n, H)
    lse = torch.logsumexp(s, -1)
    w = torch.exp(s - torch.where(lse == -math.inf, 0.0, lse)[..., None])
    o = torch.einsum("nhgm,mhd->nhgd", w, v)
    a = torch.einsum("nhgm,mhd->nhgd", w, v.abs())
    return (o.reshape(n, H, d), lse.reshape(n, H), a.reshape(n, H, d),
            size.amax(-1).reshape(n, H).double())


def attention_bounds(o, lse, a, size, d, m, v_max, e4m3):
    """Largest |error| of o [n, H, d] and lse [n, H] (64-bit values, with attention64's a and
    size).  Scores: d products summed in fp32, then the exponent's multiply-add and ex2 (2^-22):
    delta relative error of every p, once in the numerator and once in the sum.  P: one rounding
    (bf16; fp16 for e4m3, and below 2^-14 half of fp16's smallest step for each of m keys, where
    the largest p is at least 1).  O: one rounding."""
    delta = (d + 8) * F32 * (size + lse.abs().nan_to_num(0, 0, 0)) + 2.0 ** -20
    p = F16 if e4m3 else BF16
    o_tol = BF16 * o.abs() * (1 + 2.0 ** -6) + (p + 2 * delta[..., None]) * a
    if e4m3:
        o_tol = o_tol + m * 2.0 ** -25 * v_max
    return o_tol + 1e-30, 2 * delta + 2 * F32 * lse.abs().nan_to_num(0, 0, 0)


class Step:
    """A step's batch on the GPU over pages whose unused places hold NaN: q_lens new tokens and
    kv_lens lengths a sequence, `pad` rows past the last sequence, values from `seed`."""

    def __init__(self, q_lens, kv_lens, Hq, Hkv, d, page, e4m3=False, seed=0, pad=0, spare=2,
                 layout="pages", k_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.q_lens, self.kv_lens, self.page, self.d = list(q_lens), list(kv_lens), page, d
        self.Hq, self.Hkv, self.e4m3 = Hq, Hkv, e4m3
        self.S, self.T = len(q_lens), sum(q_lens) + pad
        need = [-(-n // page) for n in kv_lens]
        n_pages = sum(need) + spare
        order = torch.randperm(n_pages, generator=g).tolist()
        width = max(need + [1]) + 1
        # entries past a sequence's length are never read: they name no page
        table = torch.full((self.S, width), -7, dtype=torch.int32)
        at = 0
        for s, n in enumerate(need):
            table[s, :n] = torch.tensor(order[at:at + n], dtype=torch.int32)
            at += n
        self.table_cpu, self.table = table, table.cuda()
        starts = [sum(q_lens[:i]) for i in range(self.S + 1)]
        self.q_start = torch.tensor(starts, dtype=torch.int32).cuda()
        self.kv_len = torch.tensor(self.kv_lens, dtype=torch.int32).cuda()
        dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
        self.kd, self.vd = (0.0625, 0.125) if e4m3 else (1.0, 1.0)
        self.k64, self.v64, pages = [], [], []
        for ds, store, size in ((self.kd, self.k64, k_scale), (self.vd, self.v64, 1.0)):
            flat = torch.full((n_pages, Hkv, page, d), float("nan"))
            for s, n in enumerate(self.kv_lens):
                x = (torch.randn(n, Hkv, d, generator=g) * size / ds).to(dtype)
                store.append(x.double() * ds)
                for j0 in range(0, n, page):
                    j1 = min(n, j0 + page)
                    flat[table[s, j0 // page], :, :j1 - j0] = x[j0:j1].float().transpose(0, 1)
            pages.append(flat.to(dtype))
        if layout == "rows":  # [n_pages][page][H_kv][d] underneath
            pages = [x.transpose(1, 2).contiguous().cuda().transpose(1, 2) for x in pages]
        elif layout == "joint":  # one tensor [n_pages][2][H_kv][page][d]
            both = torch.stack([x.view(torch.uint8) for x in pages], 1).cuda().view(dtype)
            pages = [both[:, 0], both[:, 1]]
        else:
            pages = [x.cuda() for x in pages]
        self.k_pages, self.v_pages = pages
        self.q_cpu = torch.randn(self.T, Hq, d, generator=g).to(torch.bfloat16)
        self.q = self.q_cpu.cuda()
        self.max_q = max(q_lens + [0]) if isinstance(q_lens, list) else max(q_lens, default=0)

    def handles(self, max_q_len=None):
        import exact_attention_27_gb300 as fa
        return (fa.PagedCache(self.k_pages, self.v_pages, self.kd, self.vd),
                fa.PagedBatch(self.table, self.q_start, self.kv_len,
                              self.max_q if max_q_len is None else max_q_len))

    def check(self, o, lse, scale, causal, only=None):
        o, lse = o.cpu(), lse.cpu()
        t = 0
        for s, (n, m) in enumerate(zip(self.q_lens, self.kv_lens)):
            if n and (only is None or s in only):
                ro, rl, a, size = attention64(self.q_cpu[t:t + n].double(), self.k64[s],
                                              self.v64[s], scale, causal, m - n)
                vm = self.v64[s].abs().max().item() if m else 0.0
                ot, lt = attention_bounds(ro, rl, a, size, self.d, m, vm, self.e4m3)
                got, gl = o[t:t + n].double(), lse[t:t + n].double()
                empty = rl == -math.inf
                assert torch.equal(gl == -math.inf, empty), f"sequence {s}: rows without keys"
                assert torch.all(got[empty] == 0), f"sequence {s}: o of rows without keys"
                err = (got - ro).abs()
                assert torch.isfinite(got).all(), f"sequence {s}: o not finite"
                assert torch.all(err <= ot), \
                    f"sequence {s}: o off by {(err / ot).max().item():.2f} of the bound"
                lerr = (gl - rl).abs()[~empty]
                assert torch.all(lerr <= lt[~empty]), \
                    f"sequence {s}: lse off by {(lerr / lt[~empty]).max().item():.2f} of the bound"
            t += n
