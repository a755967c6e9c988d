"""What is measured of the operators around a paged key/value cache: rotary
positions with several axes, appending to the cache, and the attention of new
tokens over it.

A case is a dict of plain values.  Its batch (how many new tokens each sequence
brings and how long it is) follows from the case alone; the values follow from
the seed.  `run` computes an operator in its plain form, in elementary torch
operations, or, where `own` is true, through the library's calls.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0


# ------------------------------------------------------------------ cases

def _rotary(name, direction, B, Hq, Hkv, N, d, axes=1, rot=None, interleaved=False, fused=False):
    return {"name": name, "op": "rotary", "direction": direction, "B": B, "Hq": Hq, "Hkv": Hkv,
            "N": N, "d": d, "axes": axes, "rot": rot or d, "interleaved": interleaved,
            "fused": fused}


def _append(name, S, q_min, q_max, past_max, Hq, Hkv, d, page, cache, axes=1, batch=1, rot=None):
    return {"name": name, "op": "append", "S": S, "q_min": q_min, "q_max": q_max,
            "past_max": past_max, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "cache": cache,
            "axes": axes, "batch": batch, "rot": rot or d}


def _attention(name, S, q_min, q_max, past_min, past_max, Hq, Hkv, d, page, cache, chunks=None,
               batch=1):
    return {"name": name, "op": "attention", "S": S, "q_min": q_min, "q_max": q_max,
            "past_min": past_min, "past_max": past_max, "Hq": Hq, "Hkv": Hkv, "d": d,
            "page": page, "cache": cache, "chunks": S if chunks is None else chunks,
            "batch": batch}


def listed():
    return [
        # The training step at d = 64: q and k turned before the attention, text positions.
        _rotary("rotary_train_d64", "forward", 2, 8, 8, 4096, 64),
        # The gradient of the same for grouped heads at d = 128 over a long clip: time, height,
        # width.
        _rotary("rotary_grad_video_d128", "backward", 1, 32, 8, 16384, 128, axes=3),
        # An image of 25 x 41 patches between text, q and k as slices of one projection.
        _rotary("rotary_image_d96", "forward", 1, 16, 16, 1025, 96, axes=2, rot=64,
                interleaved=True, fused=True),
        # One new token for each of four users: the smallest call of a server.
        _append("append_token_s4", 4, 1, 1, 2000, 32, 8, 128, 16, "bf16"),
        # A prefill step over several prompts, with pictures in them, into an 8-bit cache.
        _append("append_prompts_e4m3", 7, 600, 2100, 4000, 32, 8, 128, 64, "e4m3", axes=3),
        # One new token for each of two users with short histories: latency.
        _attention("decode_s2_short", 2, 1, 1, 300, 1100, 32, 8, 128, 16, "bf16"),
        # A full server: 64 users with histories of all lengths.
        _attention("decode_s64_ragged", 64, 1, 1, 100, 8000, 32, 8, 128, 16, "bf16"),
        # One user's question about a book, 8-bit cache.
        _attention("decode_s1_long_e4m3", 1, 1, 1, 120000, 120000, 32, 8, 128, 64, "e4m3"),
        # A chunk of a long prompt behind what was cached before.
        _attention("chunk_2048_behind_30000", 1, 2048, 2048, 30000, 30000, 32, 8, 128, 64, "bf16"),
        # A scheduler's step: three chunks of prompts among 21 users' single tokens.
        _attention("mixed_s24_d64", 24, 200, 700, 1, 5000, 16, 4, 64, 32, "bf16", chunks=3),
        # Chunks of several users, 8-bit cache, a group of five query heads.
        _attention("chunks_s5_e4m3", 5, 100, 1300, 500, 7000, 20, 4, 128, 128, "e4m3"),
        # Short guesses checked against the history at head dimension 256.
        _attention("verify_s9_d256", 9, 3, 9, 200, 6000, 16, 4, 256, 16, "bf16"),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    d = rng.choice((64, 96, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    G = rng.choice((1, 2, 3, 4, 5, 7, 8))
    if Hkv * G > 32:
        G = 32 // Hkv
    op = rng.choice(("rotary", "append", "attention", "attention"))
    page = rng.choice((16, 32, 64, 128, 256))
    cache = rng.choice(("bf16", "bf16", "e4m3"))
    if op == "rotary":
        rot = rng.choice((d, d, d // 2))
        N = _log(rng, 1, 16384)
        # the largest listed case has 16384 x 40 rows of 128 values
        B = max(1, min(rng.randint(1, 4), 16384 * 40 * 128 // (N * Hkv * (G + 1) * d)))
        c = _rotary("", rng.choice(("forward", "backward")), B, Hkv * G, Hkv, N, d,
                    rng.randint(1, 3), rot, rng.random() < 0.3, rng.random() < 0.4)
    elif op == "append":
        S = _log(rng, 1, 64)
        q_max = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 8192 // S))
        c = _append("", S, max(1, q_max // 3), q_max, _log(rng, 1, 8000), Hkv * G, Hkv, d, page,
                    cache, rng.randint(1, 3), rng.randrange(1 << 20), rng.choice((d, d // 2)))
    else:
        S = _log(rng, 1, 64)
        kind = rng.choice(("decode", "verify", "chunk", "mixed"))
        q_max = {"decode": 1, "verify": rng.randint(2, 16)}.get(kind) or _log(rng, 17, 2048)
        if kind in ("chunk", "mixed"):
            S = min(S, 24 if kind == "mixed" else 6)
        past_max = _log(rng, 1, 120000)
        # no more of a cache than 64 x 8000 tokens of 8 heads, and no more products than
        # 2048 x 32000 of 32 heads, padded to the longest
        past_max = min(past_max, 64 * 8000 * 8 * 128 // (S * Hkv * d))
        past_max = max(1, min(past_max, 2048 * 32000 * 32 * 128 // (S * q_max * Hkv * G * d) - q_max))
        chunks = max(1, S // 5) if kind == "mixed" else S
        c = _attention("", S, max(1, q_max // 4), q_max, max(1, past_max // 10), past_max,
                       Hkv * G, Hkv, d, page, cache, chunks, rng.randrange(1 << 20))
    del c["name"]
    return c


def _lengths(c):
    """New tokens and length after them of each sequence: of the case alone."""
    r = random.Random(c["batch"])
    drawn = [(r.randint(c["q_min"], c["q_max"]), r.randint(c.get("past_min", 0), c["past_max"]))
             for _ in range(c["S"])]
    new = [n if s < c.get("chunks", c["S"]) else 1 for s, (n, _) in enumerate(drawn)]
    return new, [n + past for n, (_, past) in zip(new, drawn)]


def _sections(rot, axes):
    """Pairs of each axis: about a quarter for time, the rest shared by height and width."""
    half = rot // 2
    if axes == 1:
        return (half,)
    if axes == 2:
        return (half // 2, half - half // 2)
    t = half // 4
    h = (half - t) // 2
    return (t, h, half - t - h)


# ------------------------------------------------------------------ inputs

def _normal(shape, seed, dtype=torch.bfloat16):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).to(torch.float32).cuda()


def _positions(axes, shape, seed):
    """Time runs on; height and width are places in a frame."""
    n = shape[-1]
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    start = torch.randint(0, 20000, shape[:-1] + (1,), generator=g, device="cuda")
    t = torch.arange(n, device="cuda").expand(shape) + start
    by_axis = [t if axes == 1 else t // 64 + start, t % 64 // 8, t % 8]
    return torch.stack(by_axis[:axes]).to(torch.int32).contiguous()


class _State:
    pass


def prepare(case, seed):
    st = _inputs(case, seed)
    if own:
        _handles(st)
    return st


def _inputs(c, seed):
    st = _State()
    st.case = c
    d, Hq, Hkv = c["d"], c["Hq"], c["Hkv"]
    st.scale = 1.0 / math.sqrt(d)
    if c["op"] == "rotary":
        B, N = c["B"], c["N"]
        if c["fused"]:
            # slices of one projection's output [B][N][(Hq + 2 Hkv) d]
            x = _normal((B, N, Hq + 2 * Hkv, d), seed)
            st.q = x[:, :, :Hq].transpose(1, 2)
            st.k = x[:, :, Hq:Hq + Hkv].transpose(1, 2)
        else:
            st.q = _normal((B, Hq, N, d), seed)
            st.k = _normal((B, Hkv, N, d), seed + 7919)
        st.inv_freq = _inv_freq(c["rot"])
        st.positions = _positions(c["axes"], (B, N), seed + 1)
        return st

    new, total = _lengths(c)
    S, T, page = c["S"], sum(new), c["page"]
    per_seq = [-(-n // page) for n in total]
    n_pages = sum(per_seq) + 3
    st.new_max, st.total_max = max(new), max(total)
    st.q_start = torch.tensor([sum(new[:s]) for s in range(S + 1)], dtype=torch.int32,
                              device="cuda")
    st.kv_len = torch.tensor(total, dtype=torch.int32, device="cuda")
    # pages as a server hands them out: in no order
    order = list(range(n_pages))
    random.Random(seed).shuffle(order)
    ends = [sum(per_seq[:s + 1]) for s in range(S)]
    st.table = torch.tensor([order[e - n:e] + [0] * (max(per_seq) - n)
                             for n, e in zip(per_seq, ends)], dtype=torch.int32, device="cuda")
    shape = (n_pages, Hkv, page, d)
    dtype = torch.bfloat16 if c["cache"] == "bf16" else torch.float8_e4m3fn
    # an 8-bit cache holds value / descale
    st.k_descale, st.v_descale = (1.0, 1.0) if c["cache"] == "bf16" else (0.0625, 0.03125)
    st.k_pages = _pages(shape, seed + 2, dtype, st.k_descale)
    st.v_pages = _pages(shape, seed + 3, dtype, st.v_descale)
    # slices of one projection's output [T][(Hq + 2 Hkv) d]
    x = _normal((T, Hq + 2 * Hkv, d), seed)
    st.q, st.k, st.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    st.q_out = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    st.lse = torch.zeros((T, Hq), dtype=torch.float32, device="cuda")
    if c["op"] == "append":
        st.inv_freq = _inv_freq(c["rot"])
        st.positions = _positions(c["axes"], (T,), seed + 1)
    return st


def _handles(st):
    """What a program keeps for the library's calls: of a model (its rotary positions), of a
    layer (its cache), of a step (its batch), and a workspace."""
    import exact_attention_27_gb300 as fa
    c = st.case
    st.fa = fa
    if c["op"] != "attention":
        st.rotary = fa.Rotary(st.inv_freq, _sections(c["rot"], c["axes"]),
                              c.get("interleaved", False))
    if c["op"] != "rotary":
        st.cache = fa.PagedCache(st.k_pages, st.v_pages, st.k_descale, st.v_descale)
        st.batch = fa.PagedBatch(st.table, st.q_start, st.kv_len, max_q_len=st.new_max)
    if c["op"] == "attention":
        st.workspace = fa.paged_workspace(st.cache, st.batch, st.q)


def _pages(shape, seed, dtype, descale):
    x = _normal(shape, seed, torch.float32)
    return x.to(dtype) if dtype is torch.bfloat16 else (x / descale).clamp(
        -E4M3_MAX, E4M3_MAX).to(dtype)


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    op = state.case["op"]
    if op == "rotary":
        return _plain_rotary(state)
    return _plain_append(state) if op == "append" else _plain_attention(state)


def _own(st):
    c = st.case
    if c["op"] == "rotary":
        go = st.fa.rotary_forward if c["direction"] == "forward" else st.fa.rotary_backward
        return go(st.q, st.k, st.positions, st.rotary)
    if c["op"] == "append":
        st.fa.fa_paged_append(st.cache, st.batch, st.k, st.v, st.rotary, st.positions, st.q,
                              st.q_out)
        return st.q_out, st.k_pages, st.v_pages
    st.fa.fa_forward_paged(st.cache, st.batch, st.q, st.q_out, st.lse, st.scale, True,
                           st.workspace)
    return st.q_out, st.lse


def _cos_sin(c, positions, inv_freq, sign):
    """cos and sin [..., rot / 2] of every position (angles in 64 bits)."""
    axis = torch.repeat_interleave(
        torch.arange(c["axes"], device="cuda"),
        torch.tensor(_sections(c["rot"], c["axes"]), device="cuda"),
        output_size=c["rot"] // 2)
    a = positions.to(torch.float64)[axis].movedim(0, -1) * inv_freq.to(torch.float64)
    return torch.cos(a).to(torch.float32), sign * torch.sin(a).to(torch.float32)


def _turn(x, cos, sin, rot, interleaved):
    """x [..., d] in 32 bits, turned by the angles (broadcast over the heads)."""
    head, rest = x[..., :rot], x[..., rot:]
    if interleaved:
        a, b = head[..., 0::2], head[..., 1::2]
        head = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
    else:
        a, b = head[..., :rot // 2], head[..., rot // 2:]
        head = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
    return torch.cat((head, rest), -1)


def _plain_rotary(st):
    c = st.case
    cos, sin = _cos_sin(c, st.positions, st.inv_freq, 1.0 if c["direction"] == "forward" else -1.0)
    cos, sin = cos[:, None], sin[:, None]
    return tuple(_turn(x.float(), cos, sin, c["rot"], c["interleaved"]).to(torch.bfloat16)
                 for x in (st.q, st.k))


def _places(st, T):
    """Sequence, and position in it, of every new token."""
    t = torch.arange(T, device="cuda")
    start = st.q_start.long()
    s = torch.searchsorted(start[1:].contiguous(), t, right=True)
    return s, (st.kv_len.long() - start[1:])[s] + t


def _to_cache(x, st, descale):
    if st.k_pages.dtype is torch.bfloat16:
        return x.to(torch.bfloat16)
    return (x / descale).clamp(-E4M3_MAX, E4M3_MAX).to(st.k_pages.dtype)


def _plain_append(st):
    c = st.case
    cos, sin = _cos_sin(c, st.positions, st.inv_freq, 1.0)
    cos, sin = cos[:, None], sin[:, None]
    q = _turn(st.q.float(), cos, sin, c["rot"], False)
    k = _turn(st.k.float(), cos, sin, c["rot"], False)
    s, j = _places(st, st.q.shape[0])
    page, row = st.table.long()[s, j // c["page"]], j % c["page"]
    st.q_out.copy_(q.to(torch.bfloat16))
    # (8-bit pages are written through their bytes)
    bytes_of = lambda x: x if x.dtype is torch.bfloat16 else x.view(torch.uint8)  # noqa: E731
    bytes_of(st.k_pages)[page, :, row] = bytes_of(_to_cache(k, st, st.k_descale))
    bytes_of(st.v_pages)[page, :, row] = bytes_of(_to_cache(st.v.float(), st, st.v_descale))
    return st.q_out, st.k_pages, st.v_pages


def _gathered(pages, table, n, descale):
    """Every sequence's rows in order, [S, Hkv, n, d] in 32 bits."""
    S, Hkv, d = table.shape[0], pages.shape[1], pages.shape[3]
    raw = pages if pages.dtype is torch.bfloat16 else pages.view(torch.uint8)
    x = raw[table.long()].view(pages.dtype).float()
    return x.transpose(1, 2).reshape(S, Hkv, -1, d)[:, :, :n] * descale


def _plain_attention(st):
    c = st.case
    S, Hq, Hkv, d = c["S"], c["Hq"], c["Hkv"], c["d"]
    T, Q, K, G = st.q.shape[0], st.new_max, st.total_max, Hq // Hkv
    k = _gathered(st.k_pages, st.table, K, st.k_descale)
    v = _gathered(st.v_pages, st.table, K, st.v_descale)
    start = st.q_start.long()
    i = torch.arange(Q, device="cuda")
    tokens = (start[:-1, None] + i).clamp(max=T - 1)
    q = st.q[tokens].float().view(S, Q, Hkv, G, d).transpose(1, 2).reshape(S, Hkv, Q * G, d)
    scores = (q @ k.transpose(2, 3)).mul_(st.scale).view(S, Hkv, Q, G, K)
    last = st.kv_len.long() - (start[1:] - start[:-1])
    hidden = torch.arange(K, device="cuda") > (last[:, None] + i)[:, :, None]
    scores.masked_fill_(hidden[:, None, :, None], -math.inf)
    m = scores.amax(-1, keepdim=True)
    p = scores.sub_(m).exp_()
    total = p.sum(-1, keepdim=True)
    o = (p.view(S, Hkv, Q * G, K) @ v).view(S, Hkv, Q, G, d) / total
    lse = (m + total.log()).squeeze(-1)
    s, j = _places(st, T)
    at = j - last[s]
    o = o.transpose(1, 2).reshape(S, Q, Hq, d)[s, at]
    lse = lse.transpose(1, 2).reshape(S, Q, Hq)[s, at]
    return o.to(torch.bfloat16), lse


# ------------------------------------------------------------------ floors

def work(case):
    """Bytes that have to be read and written once, and operations."""
    c = case
    d, Hq, Hkv = c["d"], c["Hq"], c["Hkv"]
    if c["op"] == "rotary":
        values = c["B"] * c["N"] * (Hq + Hkv) * d
        return {"bytes": 4 * values + 4 * c["axes"] * c["B"] * c["N"], "flops": 3 * values}
    new, total = _lengths(c)
    T = sum(new)
    elem = 2 if c["cache"] == "bf16" else 1
    if c["op"] == "append":
        return {"bytes": T * d * (4 * Hq + 4 * Hkv + 2 * Hkv * elem) + 4 * c["axes"] * T,
                "flops": 3 * T * (Hq + Hkv) * d}
    pairs = sum(n * (t - n) + n * (n + 1) // 2 for n, t in zip(new, total))
    return {"bytes": 4 * T * Hq * d + 4 * T * Hq + 2 * sum(total) * Hkv * d * elem,
            "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------ in 64 bits

def _exact_turn(x, positions, c, sign, interleaved):
    """x [..., H, d]; positions [axes, ...]: every pair as a complex number."""
    rot = c["rot"]
    freq = _inv_freq(rot).double()
    edges = [0]
    for n in _sections(rot, c["axes"]):
        edges.append(edges[-1] + n)
    angle = torch.cat([positions[a].double()[..., None] * freq[edges[a]:edges[a + 1]]
                       for a in range(c["axes"])], -1)
    phase = torch.polar(torch.ones_like(angle), sign * angle)[..., None, :]
    y = x.double().clone()
    if interleaved:
        z = torch.complex(y[..., 0:rot:2].clone(), y[..., 1:rot:2].clone()) * phase
        y[..., 0:rot:2], y[..., 1:rot:2] = z.real, z.imag
    else:
        z = torch.complex(y[..., :rot // 2].clone(), y[..., rot // 2:rot].clone()) * phase
        y[..., :rot // 2], y[..., rot // 2:rot] = z.real, z.imag
    return y


def exact(case, seed):
    c, st = case, _inputs(case, seed)
    if c["op"] == "rotary":
        sign = 1.0 if c["direction"] == "forward" else -1.0
        return tuple(
            _exact_turn(x.transpose(1, 2), st.positions, c, sign, c["interleaved"]).transpose(1, 2)
            for x in (st.q, st.k))
    new, total = _lengths(c)
    page = c["page"]
    table = st.table.tolist()
    if c["op"] == "append":
        q = _exact_turn(st.q, st.positions, c, 1.0, False)
        k = _exact_turn(st.k, st.positions, c, 1.0, False) / st.k_descale
        v = st.v.double() / st.v_descale
        kp, vp = st.k_pages.double(), st.v_pages.double()
        if c["cache"] != "bf16":
            k, v = k.clamp(-E4M3_MAX, E4M3_MAX), v.clamp(-E4M3_MAX, E4M3_MAX)
        t = 0
        for s in range(c["S"]):
            j, end = total[s] - new[s], total[s]
            while j < end:
                n = min(end - j, page - j % page)
                p, r = table[s][j // page], j % page
                kp[p, :, r:r + n] = k[t:t + n].transpose(0, 1)
                vp[p, :, r:r + n] = v[t:t + n].transpose(0, 1)
                j, t = j + n, t + n
        return q, kp, vp
    o = torch.empty(st.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.empty(st.q.shape[:2], dtype=torch.float64, device="cuda")
    G, t = c["Hq"] // c["Hkv"], 0
    for s in range(c["S"]):
        n, past = new[s], total[s] - new[s]
        rows = torch.tensor(table[s][:-(-total[s] // page)], device="cuda")
        for h in range(c["Hkv"]):
            k = st.k_pages[:, h][rows] if c["cache"] == "bf16" else _bytes_rows(st.k_pages, h, rows)
            v = st.v_pages[:, h][rows] if c["cache"] == "bf16" else _bytes_rows(st.v_pages, h, rows)
            k = k.double().reshape(-1, c["d"])[:total[s]] * st.k_descale
            v = v.double().reshape(-1, c["d"])[:total[s]] * st.v_descale
            for a in range(0, n, 512):
                b = min(n, a + 512)
                x = st.q[t + a:t + b, h * G:(h + 1) * G].double()
                logits = torch.einsum("igd,jd->igj", x, k[:past + b]) * st.scale
                see = torch.arange(past + b, device="cuda")[None, :] <= (
                    torch.arange(a, b, device="cuda") + past)[:, None]
                logits = logits.masked_fill(~see[:, None], -math.inf)
                o[t + a:t + b, h * G:(h + 1) * G] = torch.softmax(logits, -1) @ v[:past + b]
                lse[t + a:t + b, h * G:(h + 1) * G] = torch.logsumexp(logits, -1)
        t += n
    return o, lse


def _bytes_rows(pages, h, rows):
    return pages.view(torch.uint8)[:, h][rows].view(pages.dtype)
