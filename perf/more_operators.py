"""What is measured of attention whose scores are shaped (capped by a tanh, lowered with the
distance, seen through documents, prefixes, windows and padding), trained and served, and of the
norms of each head's queries and keys that go with the position rotation.

A case is a dict of plain values.  Its masks and its batch (documents, prefixes, how many new
tokens each sequence brings) follow from the case alone; the values follow from the seed.  `run`
computes an operator in its plain form, in elementary torch operations, or, where `own` is true,
through the library's calls.
"""

import math
import random

import torch

own = False

E4M3_MAX = 448.0
EPS = 1e-6


# ------------------------------------------------------------------ cases

def _norm(name, direction, B, Hq, Hkv, N, d, axes=1, rot=None, interleaved=False, fused=False,
          weights="fp32"):
    return {"name": name, "op": "norm", "direction": direction, "B": B, "Hq": Hq, "Hkv": Hkv,
            "N": N, "d": d, "axes": axes, "rot": rot or d, "interleaved": interleaved,
            "fused": fused, "weights": weights}


def _append(name, S, q_min, q_max, past_max, Hq, Hkv, d, page, cache, axes=1, batch=1, rot=None,
            weights="fp32"):
    return {"name": name, "op": "append", "S": S, "q_min": q_min, "q_max": q_max,
            "past_max": past_max, "Hq": Hq, "Hkv": Hkv, "d": d, "page": page, "cache": cache,
            "axes": axes, "batch": batch, "rot": rot or d, "weights": weights}


def _scores(name, direction, B, Hq, Hkv, Nq, d, mask, Nkv=None, cap=0.0, slopes=False, window=0,
            batch=1):
    return {"name": name, "op": "scores", "direction": direction, "B": B, "Hq": Hq, "Hkv": Hkv,
            "Nq": Nq, "Nkv": Nkv or Nq, "d": d, "mask": mask, "cap": cap, "slopes": slopes,
            "window": window, "batch": batch}


def _paged(name, S, q_min, q_max, past_min, past_max, Hq, Hkv, d, page, cache, cap=0.0,
           slopes=False, window=0, batch=1):
    return {"name": name, "op": "paged", "S": S, "q_min": q_min, "q_max": q_max,
            "past_min": past_min, "past_max": past_max, "Hq": Hq, "Hkv": Hkv, "d": d,
            "page": page, "cache": cache, "cap": cap, "slopes": slopes, "window": window,
            "batch": batch}


def listed():
    return [
        # The training step at d = 64: q and k normed and turned before the attention.
        _norm("norm_train_d64", "forward", 2, 8, 8, 4096, 64),
        # The gradient of the same for grouped heads at d = 128 over a clip, slices of one
        # projection: of q, of k and of both norms' weights.
        _norm("norm_grad_video_d128", "backward", 1, 32, 8, 8192, 128, axes=3, fused=True,
              weights="bf16"),
        # One new token for each of four users: the smallest call of a server.
        _append("append_norm_token_s4", 4, 1, 1, 2000, 32, 8, 128, 16, "bf16"),
        # A prefill step over several prompts into an 8-bit cache.
        _append("append_norm_prompts_e4m3", 7, 600, 2100, 4000, 32, 8, 128, 64, "e4m3"),
        # A short prompt whose beginning is seen by all of it, scores capped: latency.
        _scores("prefix_short_d64", "forward", 1, 4, 2, 77, 64, "prefix", cap=50.0),
        # The training step at d = 64 on packed documents, the last rows padding.
        _scores("packed_train_d64", "train", 2, 8, 8, 4096, 64, "documents"),
        # A long training step with capped scores and grouped heads.
        _scores("cap_train_d128", "train", 1, 16, 4, 8192, 128, "causal", cap=50.0),
        # Scores that fall with the distance, at a length that fills no tile.
        _scores("slopes_forward_d96", "forward", 1, 16, 16, 5001, 96, "causal", slopes=True),
        # A layer with a window and capped scores at head dimension 256, trained.
        _scores("window_train_d256", "train", 1, 8, 4, 4000, 256, "causal", cap=50.0, window=1024),
        # One new token for each of 64 users, scores capped, in a layer with a window.
        _paged("decode_window_s64", 64, 1, 1, 100, 8000, 32, 8, 128, 16, "bf16", cap=50.0,
               window=4096),
        # One new token for each of three users, scores that fall with the distance: latency.
        _paged("decode_slopes_s3", 3, 1, 1, 300, 1100, 16, 4, 64, 16, "bf16", slopes=True),
        # A chunk of a long prompt behind what was cached before, capped, 8-bit cache.
        _paged("chunk_cap_e4m3", 1, 1024, 1024, 15000, 15000, 32, 8, 128, 64, "e4m3", cap=50.0),
    ]


def _log(rng, a, b):
    return int(round(math.exp(rng.uniform(math.log(a), math.log(b)))))


def draw(rng):
    d = rng.choice((64, 96, 128, 128, 256))
    Hkv = rng.choice((1, 2, 4, 5, 8))
    G = rng.choice((1, 2, 3, 4, 5, 7, 8))
    if Hkv * G > 32:
        G = 32 // Hkv
    op = rng.choice(("norm", "append", "scores", "scores", "scores", "paged", "paged"))
    page = rng.choice((16, 32, 64, 128, 256))
    cache = rng.choice(("bf16", "bf16", "e4m3"))
    weights = rng.choice(("fp32", "bf16"))
    cap = rng.choice((0.0, round(rng.uniform(15.0, 60.0), 1)))
    slopes = rng.random() < 0.4
    batch = rng.randrange(1 << 20)
    if op == "norm":
        N = _log(rng, 1, 16384)
        # the largest listed case has 8192 x 40 rows of 128 values
        B = max(1, min(rng.randint(1, 4), 8192 * 40 * 128 // (N * Hkv * (G + 1) * d)))
        N = max(1, min(N, 8192 * 40 * 128 // (B * Hkv * (G + 1) * d)))
        c = _norm("", rng.choice(("forward", "backward")), B, Hkv * G, Hkv, N, d,
                  rng.randint(1, 3), rng.choice((d, d, d // 2)), rng.random() < 0.3,
                  rng.random() < 0.4, weights)
    elif op == "append":
        S = _log(rng, 1, 64)
        q_max = 1 if rng.random() < 0.4 else _log(rng, 2, max(2, 8192 // S))
        c = _append("", S, max(1, q_max // 3), q_max, _log(rng, 1, 8000), Hkv * G, Hkv, d, page,
                    cache, rng.randint(1, 3), batch, rng.choice((d, d // 2)), weights)
    elif op == "scores":
        mask = rng.choice(("causal", "documents", "prefix", "padded", "full", "behind"))
        Nq = _log(rng, 1, 8192)
        # no more products than those of 16 causal heads of 8192 positions
        most = 16 * 8192 * 8192 * 128 // (Hkv * G * d)
        if mask not in ("causal", "documents"):
            most //= 2
        B = max(1, min(rng.randint(1, 4), most // (Nq * Nq)))
        Nq = min(Nq, math.isqrt(most // B))
        Nkv = Nq
        if mask == "behind":
            Nkv = Nq + _log(rng, 1, max(1, min(8192, most // (B * Nq) - Nq)))
        window = _log(rng, 1, Nkv) if mask in ("causal", "documents", "behind") and \
            rng.random() < 0.4 else 0
        c = _scores("", rng.choice(("forward", "train")), B, Hkv * G, Hkv, Nq, d, mask, Nkv, cap,
                    slopes, window, batch)
    else:
        S = _log(rng, 1, 64)
        kind = rng.choice(("decode", "verify", "chunk"))
        q_max = {"decode": 1, "verify": rng.randint(2, 16)}.get(kind) or _log(rng, 17, 1024)
        if kind == "chunk":
            S = min(S, 6)
        past_max = _log(rng, 1, 60000)
        # no more of a cache than 64 x 3300 tokens of 8 heads, and no more products than
        # 1024 x 16024 of 32 heads, padded to the longest
        past_max = min(past_max, 64 * 3300 * 8 * 128 // (S * Hkv * d))
        past_max = max(1, min(past_max, 1024 * 16024 * 32 * 128 // (S * q_max * Hkv * G * d) - q_max))
        window = _log(rng, 1, past_max + q_max) if rng.random() < 0.5 else 0
        c = _paged("", S, max(1, q_max // 4), q_max, max(1, past_max // 10), past_max, Hkv * G,
                   Hkv, d, page, cache, cap, slopes, window, batch)
    del c["name"]
    return c


def _lengths(c):
    """New tokens and length after them of each sequence: of the case alone."""
    r = random.Random(c["batch"])
    new = [r.randint(c["q_min"], c["q_max"]) for _ in range(c["S"])]
    return new, [n + r.randint(c.get("past_min", 0), c["past_max"]) for n in new]


def _spans(c):
    """First and end of the keys that each query may see, a row for each batch entry (None: from
    the first, to the last), before the causal mask and the window: of the case alone."""
    r = random.Random(c["batch"])
    N = c["Nq"]
    first, end = [], []
    for _ in range(c["B"]):
        if c["mask"] == "documents":
            f, e = [], []
            real = N - int(N * r.uniform(0.0, 0.05))  # rows past it are padding and see nothing
            while len(f) < real:
                n = min(real - len(f), max(1, int(round(math.exp(r.uniform(
                    math.log(max(1.0, N / 40)), math.log(max(1.0, N / 2))))))))
                a = len(f)
                f += [a] * n
                e += [a + n] * n
            first.append(f + [0] * (N - real))
            end.append(e + [0] * (N - real))
        elif c["mask"] == "prefix":
            p = r.randint(0, N)
            end.append([max(i + 1, p) for i in range(N)])
        elif c["mask"] == "padded":
            end.append([r.randint((N + 1) // 2, N)] * N)
    return first or None, end or None


def _seen(c, b, spans):
    """First and end, as lists, of the keys that the queries of batch entry b see after all."""
    first, end = spans
    off = c["Nkv"] - c["Nq"]
    lo = list(first[b]) if first else [0] * c["Nq"]
    hi = list(end[b]) if end else [c["Nkv"]] * c["Nq"]
    if c["mask"] in ("causal", "documents", "behind"):
        hi = [min(h, off + i + 1) for i, h in enumerate(hi)]
    if c["window"]:
        lo = [max(a, off + i + 1 - c["window"]) for i, a in enumerate(lo)]
    return lo, hi


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

def _normal(shape, seed, dtype=torch.bfloat16, gain=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(int(seed))
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).mul_(gain).to(dtype)


def _weight(c, seed):
    """A norm's weight, near 1 as training leaves it."""
    w = 1.0 + 0.2 * _normal((c["d"],), seed, torch.float32)
    return w if c["weights"] == "fp32" else w.to(torch.bfloat16)


def _inv_freq(rot):
    i = torch.arange(rot // 2, dtype=torch.float64)
    return (10000.0 ** (-2.0 * i / rot)).to(torch.float32).cuda()


def _slopes(Hq):
    h = torch.arange(1, Hq + 1, dtype=torch.float64)
    return (2.0 ** (-8.0 * h / Hq)).to(torch.float32).cuda()


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
    if c["op"] in ("norm", "append"):
        st.inv_freq = _inv_freq(c["rot"])
        st.qw, st.kw = _weight(c, seed + 11), _weight(c, seed + 12)
    if c["op"] == "norm":
        B, N = c["B"], c["N"]
        st.positions = _positions(c["axes"], (B, N), seed + 1)
        if c["fused"]:
            # slices of one projection's output [B][N][(Hq + 2 Hkv) d]
            x = _normal((B, N, Hq + 2 * Hkv, d), seed, gain=2.0)
            st.q = x[:, :, :Hq].transpose(1, 2)
            st.k = x[:, :, Hq:Hq + Hkv].transpose(1, 2)
        else:
            st.q = _normal((B, Hq, N, d), seed, gain=2.0)
            st.k = _normal((B, Hkv, N, d), seed + 7919, gain=2.0)
        if c["direction"] == "backward":
            st.dq = _normal((B, Hq, N, d), seed + 21)
            st.dk = _normal((B, Hkv, N, d), seed + 22)
        return st
    if c["op"] == "scores":
        B = c["B"]
        # (scores of a trained model: a standard deviation of two)
        st.q = _normal((B, Hq, c["Nq"], d), seed, gain=2.0)
        st.k = _normal((B, Hkv, c["Nkv"], d), seed + 1)
        st.v = _normal((B, Hkv, c["Nkv"], d), seed + 2)
        if c["direction"] == "train":
            st.do = _normal((B, Hq, c["Nq"], d), seed + 3)
        first, end = _spans(c)
        st.first = torch.tensor(first, dtype=torch.int32, device="cuda") if first else None
        st.end = torch.tensor(end, dtype=torch.int32, device="cuda") if end else None
        st.slopes = _slopes(Hq) if c["slopes"] else None
        st.causal = c["mask"] in ("causal", "documents", "behind")
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
    x = _normal((T, Hq + 2 * Hkv, d), seed, gain=2.0)
    st.q, st.k, st.v = x[:, :Hq], x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:]
    st.q_out = torch.zeros((T, Hq, d), dtype=torch.bfloat16, device="cuda")
    st.lse = torch.zeros((T, Hq), dtype=torch.float32, device="cuda")
    if c["op"] == "append":
        st.positions = _positions(c["axes"], (T,), seed + 1)
    else:
        st.slopes = _slopes(Hq) if c["slopes"] else None
    return st


def _pages(shape, seed, dtype, descale):
    x = _normal(shape, seed, torch.float32)
    return x.to(dtype) if dtype is torch.bfloat16 else (x / descale).clamp(
        -E4M3_MAX, E4M3_MAX).to(dtype)


def _handles(st):
    """What a program keeps for the library's calls: of a model (its rotary positions, its norms,
    its scores), of a layer (its cache), of a step (its batch or its masks), and a workspace."""
    import exact_attention_27_gb300 as fa
    c = st.case
    st.fa = fa
    if c["op"] in ("norm", "append"):
        st.rotary = fa.Rotary(st.inv_freq, _sections(c["rot"], c["axes"]),
                              c.get("interleaved", False))
        st.norm = fa.HeadNorm(st.qw, st.kw, EPS)
    else:
        st.scores = fa.Scores(softcap=c["cap"], slopes=st.slopes, window=c["window"])
    if c["op"] == "scores":
        st.spans = fa.KeySpans(st.first, st.end) if c["mask"] in (
            "documents", "prefix", "padded") else None
    if c["op"] in ("append", "paged"):
        st.cache = fa.PagedCache(st.k_pages, st.v_pages, st.k_descale, st.v_descale)
        st.batch = fa.PagedBatch(st.table, st.q_start, st.kv_len, max_q_len=st.new_max)
    if c["op"] == "paged":
        st.workspace = fa.paged_workspace(st.cache, st.batch, st.q)


# ------------------------------------------------------------------ one pass

def run(state):
    if own:
        return _own(state)
    op = state.case["op"]
    if op == "norm":
        return _plain_norm(state)
    if op == "append":
        return _plain_append(state)
    return _plain_scores(state) if op == "scores" else _plain_paged(state)


def _own(st):
    c = st.case
    if c["op"] == "norm":
        if c["direction"] == "forward":
            return st.fa.norm_rotary_forward(st.q, st.k, st.norm, st.positions, st.rotary)
        return st.fa.norm_rotary_backward(st.dq, st.dk, st.q, st.k, st.norm, st.positions,
                                          st.rotary)
    if c["op"] == "append":
        st.fa.fa_paged_append(st.cache, st.batch, st.k, st.v, st.rotary, st.positions, st.q,
                              st.q_out, norm=st.norm)
        return st.q_out, st.k_pages, st.v_pages
    if c["op"] == "paged":
        st.fa.fa_forward_paged(st.cache, st.batch, st.q, st.q_out, st.lse, st.scale, True,
                               st.workspace, scores=st.scores)
        return st.q_out, st.lse
    shape = {"causal": st.causal, "scale": st.scale, "scores": st.scores, "spans": st.spans,
             "q_offset": c["Nkv"] - c["Nq"]}
    o, lse = st.fa.attention_forward(st.q, st.k, st.v, **shape)
    if c["direction"] == "forward":
        return o, lse
    return (o, lse) + tuple(st.fa.attention_backward(st.q, st.k, st.v, o, lse, st.do, **shape))


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


def _unit(x):
    """x in 32 bits over the root of its mean square, and one over that root."""
    x = x.float()
    r = torch.rsqrt((x * x).mean(-1, keepdim=True) + EPS)
    return x * r, r


def _plain_norm_one(c, x, w, cos, sin):
    return _turn(_unit(x)[0] * w.float(), cos, sin, c["rot"], c.get("interleaved", False))


def _plain_norm_grad(c, g, x, w, cos, sin):
    """Gradients of x and of its weight from g, that of the turned output (cos, -sin: back)."""
    g = _turn(g.float(), cos, sin, c["rot"], c["interleaved"])
    u, r = _unit(x)
    gu = g * w.float()
    dx = r * (gu - u * (gu * u).mean(-1, keepdim=True))
    # (a sum over every position: in 64 bits)
    dw = (g * u).sum(-2, dtype=torch.float64).sum((0, 1)).to(torch.float32)
    return dx.to(torch.bfloat16), dw


def _plain_norm(st):
    c = st.case
    forward = c["direction"] == "forward"
    cos, sin = _cos_sin(c, st.positions, st.inv_freq, 1.0 if forward else -1.0)
    cos, sin = cos[:, None], sin[:, None]
    if forward:
        return tuple(_plain_norm_one(c, x, w, cos, sin).to(torch.bfloat16)
                     for x, w in ((st.q, st.qw), (st.k, st.kw)))
    dq, dqw = _plain_norm_grad(c, st.dq, st.q, st.qw, cos, sin)
    dk, dkw = _plain_norm_grad(c, st.dk, st.k, st.kw, cos, sin)
    return dq, dk, dqw, dkw


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
    q = _plain_norm_one(c, st.q, st.qw, cos, sin)
    k = _plain_norm_one(c, st.k, st.kw, cos, sin)
    s, j = _places(st, st.q.shape[0])
    page, row = st.table.long()[s, j // c["page"]], j % c["page"]
    st.q_out.copy_(q.to(torch.bfloat16))
    # (8-bit pages are written through their bytes)
    bytes_of = lambda x: x if x.dtype is torch.bfloat16 else x.view(torch.uint8)  # noqa: E731
    bytes_of(st.k_pages)[page, :, row] = bytes_of(_to_cache(k, st, st.k_descale))
    bytes_of(st.v_pages)[page, :, row] = bytes_of(_to_cache(st.v.float(), st, st.v_descale))
    return st.q_out, st.k_pages, st.v_pages


def _shaped(c, s, slopes, qpos, kpos):
    """Scores [..., Hkv, G, Nq, Nkv] (written over), and the tanh that capped them (None: not
    capped).  qpos [..., Nq], kpos [Nkv]."""
    t = None
    if c["cap"]:
        t = s.div_(c["cap"]).tanh_()
        s = t * c["cap"]
    if slopes is not None:
        distance = (qpos[..., :, None] - kpos).abs().float()
        s = s.sub_(slopes.view(c["Hkv"], -1, 1, 1) * distance)
    return s, t


def _softmax(s, hidden):
    """Weights and log of their sum [..., 1]; zeros and -inf for rows that see nothing."""
    s = s.masked_fill_(hidden, -math.inf)
    m = s.amax(-1, keepdim=True)
    p = s.sub_(m.clamp(min=-3e38)).exp_()
    total = p.sum(-1, keepdim=True)
    return p.div_(total.clamp(min=1e-30)), m + total.log()


def _plain_scores(st):
    c = st.case
    B, Hq, Hkv, Nq, Nkv, d = (c[x] for x in ("B", "Hq", "Hkv", "Nq", "Nkv", "d"))
    kpos = torch.arange(Nkv, device="cuda")
    qpos = torch.arange(Nq, device="cuda") + (Nkv - Nq)
    hidden = torch.zeros((1, Nq, Nkv), dtype=torch.bool, device="cuda")
    if st.causal:
        hidden = hidden | (kpos > qpos[:, None])
    if c["window"]:
        hidden = hidden | (kpos <= qpos[:, None] - c["window"])
    if st.first is not None:
        hidden = hidden | (kpos < st.first[:, :, None])
    if st.end is not None:
        hidden = hidden | (kpos >= st.end[:, :, None])
    hidden = hidden[:, None, None]
    q = st.q.float().view(B, Hkv, -1, Nq, d)
    k, v = st.k.float()[:, :, None], st.v.float()[:, :, None]
    s, t = _shaped(c, (q @ k.transpose(-1, -2)).mul_(st.scale), st.slopes, qpos, kpos)
    p, lse = _softmax(s, hidden)
    o = p @ v
    out = o.view(B, Hq, Nq, d).to(torch.bfloat16), lse.view(B, Hq, Nq)
    if c["direction"] == "forward":
        return out
    do = st.do.float().view(B, Hkv, -1, Nq, d)
    dv = (p.transpose(-1, -2) @ do).sum(2)
    ds = (do @ v.transpose(-1, -2)).sub_((do * o).sum(-1, keepdim=True)).mul_(p)
    if t is not None:
        ds.mul_(1.0 - t * t)
    dq = (ds @ k).mul_(st.scale)
    dk = (ds.transpose(-1, -2) @ q).sum(2).mul_(st.scale)
    return out + (dq.view(B, Hq, Nq, d).to(torch.bfloat16), dk.to(torch.bfloat16),
                  dv.to(torch.bfloat16))


def _gathered(pages, table, n, descale):
    """Every sequence's rows in order, [S, Hkv, n, d] in 32 bits."""
    S, Hkv, d = table.shape[0], pages.shape[1], pages.shape[3]
    raw = pages if pages.dtype is torch.bfloat16 else pages.view(torch.uint8)
    x = raw[table.long()].view(pages.dtype).float()
    return x.transpose(1, 2).reshape(S, Hkv, -1, d)[:, :, :n] * descale


def _plain_paged(st):
    c = st.case
    S, Hq, Hkv, d = c["S"], c["Hq"], c["Hkv"], c["d"]
    T, Q, K, G = st.q.shape[0], st.new_max, st.total_max, Hq // Hkv
    k = _gathered(st.k_pages, st.table, K, st.k_descale)
    v = _gathered(st.v_pages, st.table, K, st.v_descale)
    start = st.q_start.long()
    i = torch.arange(Q, device="cuda")
    tokens = (start[:-1, None] + i).clamp(max=T - 1)
    q = st.q[tokens].float().view(S, Q, Hkv, G, d).permute(0, 2, 3, 1, 4)
    last = st.kv_len.long() - (start[1:] - start[:-1])
    qpos, kpos = last[:, None] + i, torch.arange(K, device="cuda")
    s = (q.reshape(S, Hkv, G * Q, d) @ k.transpose(2, 3)).mul_(st.scale).view(S, Hkv, G, Q, K)
    s, _ = _shaped(c, s, st.slopes, qpos[:, None, None], kpos)
    hidden = kpos > qpos[:, :, None]
    if c["window"]:
        hidden = hidden | (kpos <= qpos[:, :, None] - c["window"])
    p, lse = _softmax(s, hidden[:, None, None])
    o = (p.view(S, Hkv, G * Q, K) @ v).view(S, Hq, Q, d)
    s, j = _places(st, T)
    at = j - last[s]
    return (o.transpose(1, 2)[s, at].to(torch.bfloat16),
            lse.reshape(S, Hq, Q).transpose(1, 2)[s, at])


# ------------------------------------------------------------------ floors

def work(case):
    """Bytes that have to be read and written once, and operations."""
    c = case
    d, Hq, Hkv = c["d"], c["Hq"], c["Hkv"]
    if c["op"] == "norm":
        values = c["B"] * c["N"] * (Hq + Hkv) * d
        back = c["direction"] == "backward"
        return {"bytes": (6 if back else 4) * values + 4 * c["axes"] * c["B"] * c["N"],
                "flops": (14 if back else 7) * values}
    if c["op"] == "scores":
        spans = _spans(c)
        pairs = sum(max(0, e - f) for b in range(c["B"]) for f, e in zip(*_seen(c, b, spans)))
        q_rows, k_rows = c["B"] * Hq * c["Nq"], c["B"] * Hkv * c["Nkv"]
        if c["direction"] == "forward":
            return {"bytes": 4 * (q_rows + k_rows) * d + 4 * q_rows, "flops": 4 * pairs * Hq * d}
        # forward two products, backward four (the scores themselves could be kept)
        return {"bytes": 8 * (q_rows + k_rows) * d + 4 * q_rows, "flops": 12 * pairs * Hq * d}
    new, total = _lengths(c)
    T = sum(new)
    elem = 2 if c["cache"] == "bf16" else 1
    if c["op"] == "append":
        return {"bytes": T * d * (4 * Hq + 4 * Hkv + 2 * Hkv * elem) + 4 * c["axes"] * T,
                "flops": 7 * T * (Hq + Hkv) * d}
    w = c["window"] or max(total)
    pairs = sum(min(t - n + i + 1, w) for n, t in zip(new, total) for i in range(n))
    keys = sum(min(t, n - 1 + w) for n, t in zip(new, total))
    return {"bytes": 4 * T * Hq * d + 4 * T * Hq + 2 * keys * Hkv * d * elem,
            "flops": 4 * pairs * Hq * d}


# ------------------------------------------------------------------ in 64 bits

def _exact_turn(x, positions, c):
    """x [..., H, d] in 64 bits; positions [axes, ...]: every pair as a complex number."""
    rot = c["rot"]
    freq = _inv_freq(rot).double()
    edges = [0]
    for n in _sections(rot, c["axes"]):
        edges.append(edges[-1] + n)
    angle = torch.cat([positions[a].double()[..., None] * freq[edges[a]:edges[a + 1]]
                       for a in range(c["axes"])], -1)
    phase = torch.polar(torch.ones_like(angle), angle)[..., None, :]
    if c.get("interleaved"):
        z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * phase
        head = torch.view_as_real(z).flatten(-2)
    else:
        z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * phase
        head = torch.cat((z.real, z.imag), -1)
    return torch.cat((head, x[..., rot:]), -1)


def _exact_norm(x, w):
    return x / torch.sqrt(x.square().mean(-1, keepdim=True) + EPS) * w


def exact(case, seed):
    c, st = case, _inputs(case, seed)
    if c["op"] == "norm":
        outs, grads = [], []
        for x, w, g in ((st.q, st.qw, getattr(st, "dq", None)), (st.k, st.kw, getattr(st, "dk", None))):
            x, w = x.double().requires_grad_(g is not None), w.double().requires_grad_(g is not None)
            y = _exact_turn(_exact_norm(x, w).transpose(1, 2), st.positions, c).transpose(1, 2)
            if g is None:
                outs.append(y)
            else:
                grads.append(torch.autograd.grad(y, (x, w), g.double()))
        return tuple(outs) if outs else (grads[0][0], grads[1][0], grads[0][1], grads[1][1])
    if c["op"] == "scores":
        return _exact_scores(c, st)
    new, total = _lengths(c)
    page = c["page"]
    table = st.table.tolist()
    if c["op"] == "append":
        q = _exact_turn(_exact_norm(st.q.double(), st.qw.double()), st.positions, c)
        k = _exact_turn(_exact_norm(st.k.double(), st.kw.double()), st.positions, c) / st.k_descale
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
            k, v = (_rows(x, h, rows).double().reshape(-1, c["d"])[:total[s]] * f
                    for x, f in ((st.k_pages, st.k_descale), (st.v_pages, st.v_descale)))
            for a in range(0, n, 512):
                b = min(n, a + 512)
                lo = max(0, past + a + 1 - c["window"]) if c["window"] else 0
                key = torch.arange(lo, past + b, device="cuda")
                pos = torch.arange(past + a, past + b, device="cuda")
                x = st.q[t + a:t + b, h * G:(h + 1) * G].double()
                logits = torch.einsum("igd,jd->gij", x, k[lo:past + b]) * st.scale
                slopes = st.slopes[h * G:(h + 1) * G] if c["slopes"] else None
                logits = _exact_logits(c, logits, slopes, pos, key)
                see = key <= pos[:, None]
                if c["window"]:
                    see &= key > pos[:, None] - c["window"]
                logits = logits.masked_fill(~see, -math.inf)
                o[t + a:t + b, h * G:(h + 1) * G] = (
                    torch.softmax(logits, -1) @ v[lo:past + b]).transpose(0, 1)
                lse[t + a:t + b, h * G:(h + 1) * G] = torch.logsumexp(logits, -1).transpose(0, 1)
        t += n
    return o, lse


def _rows(pages, h, rows):
    if pages.dtype is torch.bfloat16:
        return pages[:, h][rows]
    return pages.view(torch.uint8)[:, h][rows].view(pages.dtype)


def _exact_logits(c, logits, slopes, pos, key):
    if c["cap"]:
        logits = c["cap"] * torch.tanh(logits / c["cap"])
    if slopes is not None:
        logits = logits - slopes.double()[:, None, None] * (pos[:, None] - key).abs().double()
    return logits


def _exact_scores(c, st):
    """Head after head; gradients by differentiating the forward."""
    train = c["direction"] == "train"
    G, off, spans = c["Hq"] // c["Hkv"], c["Nkv"] - c["Nq"], _spans(c)
    o = torch.zeros(st.q.shape, dtype=torch.float64, device="cuda")
    lse = torch.full(st.q.shape[:3], -math.inf, dtype=torch.float64, device="cuda")
    dq, dk, dv = (torch.zeros(x.shape, dtype=torch.float64, device="cuda")
                  for x in (st.q, st.k, st.v))
    key = torch.arange(c["Nkv"], device="cuda")
    for b in range(c["B"]):
        lo, hi = (torch.tensor(x, device="cuda") for x in _seen(c, b, spans))
        live = torch.nonzero(hi > lo)[:, 0]  # rows that see something
        if not len(live):
            continue
        see = (key >= lo[live, None]) & (key < hi[live, None])
        for h in range(c["Hq"]):
            q, k, v = (x.double().requires_grad_(train) for x in (
                st.q[b, h][live], st.k[b, h // G], st.v[b, h // G]))
            logits = (q @ k.T * st.scale)[None]
            slopes = st.slopes[h:h + 1] if c["slopes"] else None
            logits = _exact_logits(c, logits, slopes, live + off, key)[0]
            logits = logits.masked_fill(~see, -math.inf)
            y = torch.softmax(logits, -1) @ v
            o[b, h, live] = y.detach()
            lse[b, h, live] = torch.logsumexp(logits.detach(), -1)
            if train:
                g = torch.autograd.grad(y, (q, k, v), st.do[b, h][live].double())
                dq[b, h, live] = g[0]
                dk[b, h // G] += g[1]
                dv[b, h // G] += g[2]
            del q, k, v, logits, y
    return (o, lse, dq, dk, dv) if train else (o, lse)
