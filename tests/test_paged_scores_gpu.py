"""Attention with shaped scores over a paged cache, from single tokens to chunks, against 64-bit
values."""

import math

import pytest
import torch

from paged_plain import BF16, F16, Step
from scores_plain import Head, spans_of

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def alibi(H):
    return torch.tensor([2.0 ** (-8.0 * (h + 1) / H) for h in range(H)])


def attend(step, scores, causal=True, max_q_len=None, stream=None):
    import exact_attention_27_gb300 as fa
    cache, batch = step.handles(max_q_len)
    o = torch.full((step.T, step.Hq, step.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((step.T, step.Hq), float("nan"), device="cuda")
    ws = fa.paged_workspace(cache, batch, step.q)
    ws.fill_(0xFF)
    fa.fa_forward_paged(cache, batch, step.q, o, lse, 1 / math.sqrt(step.d), causal, ws, stream,
                        scores)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    used = sum(step.q_lens)
    assert torch.isnan(o[used:]).all() and torch.isnan(lse[used:]).all()
    return o, lse


def check(step, o, lse, softcap=0.0, slopes=None, window=0, causal=True):
    """Every token of every sequence against Head's values and bounds; over e4m3 pages the weights
    are fp16 (2^-11 of each, and 2^-32 of the largest, of which a row has at most m)."""
    o, lse = o.cpu().double(), lse.cpu().double()
    G, t = step.Hq // step.Hkv, 0
    for s, (n, m) in enumerate(zip(step.q_lens, step.kv_lens)):
        off = m - n
        see = spans_of(n, m, causal, off, window)
        for h in range(step.Hq if n else 0):
            x = Head(step.q_cpu[t:t + n, h].double(), step.k64[s][:, h // G], step.v64[s][:, h // G],
                     see, 1 / math.sqrt(step.d), softcap,
                     0.0 if slopes is None else float(slopes[h]), off)
            tol = x.o_tol
            if step.e4m3:
                a = (x.o_tol - BF16 * x.o.abs() * (1 + 2.0 ** -6)) / BF16 * F16
                big = step.v64[s].abs().max() if m else 0.0
                tol = BF16 * x.o.abs() * (1 + 2.0 ** -6) + a + m * 2.0 ** -25 * big + \
                    2 * x.delta[:, None] * big
            got = o[t:t + n, h]
            err = (got - x.o).abs() / tol
            assert torch.isfinite(got).all(), f"sequence {s}: o not finite"
            assert err.max() <= 1, f"sequence {s}: o off by {err.max().item():.2f} of its bound"
            gl = lse[t:t + n, h]
            assert torch.equal(gl == -math.inf, ~x.live), f"sequence {s}: rows without keys"
            el = torch.where(x.live, (gl - x.lse).abs() / x.lse_tol, torch.zeros_like(gl))
            assert el.max() <= 1, f"sequence {s}: lse off by {el.max().item():.2f} of its bound"
        t += n


KINDS = {"cap": dict(softcap=15.0), "slopes": dict(slopes=True), "window": dict(window=70),
         "all": dict(softcap=15.0, slopes=True, window=100), "window 1": dict(window=1)}


def go(step, causal=True, **kw):
    import exact_attention_27_gb300 as fa
    kw = dict(kw)
    if kw.get("slopes") is True:
        kw["slopes"] = alibi(step.Hq)
    dev = dict(kw)
    if "slopes" in dev:
        dev["slopes"] = dev["slopes"].cuda()
    o, lse = attend(step, fa.Scores(**dev), causal)
    check(step, o, lse, causal=causal, **kw)
    return o, lse


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(d, page, kind, e4m3):
    lens = [1, 15, 63, 64, 65, 127, 129, 300, 777]
    go(Step([1] * len(lens), lens, 8, 2, d, page, e4m3, seed=d + page, pad=2, k_scale=3.0),
       **KINDS[kind])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("kind", list(KINDS))
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_chunks(causal, d, kind, e4m3):
    q = [0, 1, 33, 128, 129, 5, 0, 200]
    k = [40, 700, 33, 128, 400, 6, 0, 513]
    go(Step(q, k, 6, 2, d, 32, e4m3, seed=d + causal, pad=1), causal, **KINDS[kind])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[3, 2, 4], [1, 16, 1], [300, 1, 40]])
def test_windows_over_long_histories(new, d, e4m3):
    """Windows that begin inside a page, at one, and before the sequence does; work that many CTAs
    share."""
    for window in (16, 65, 128, 1000, 5000):
        go(Step(new, [n + 4000 + 37 * i for i, n in enumerate(new)], 4, 1, d, 16, e4m3, seed=window),
           window=window, softcap=30.0)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[1, 1], [20, 150]])
@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_before_the_window_may_be_gone(new, d, e4m3):
    """Entries of the table for pages before every window name no page, and what lies before the
    window in its first page is NaN."""
    import exact_attention_27_gb300 as fa
    page, window = 32, 90
    lens = [n + 700 + i for i, n in enumerate(new)]
    step = Step(new, lens, 4, 2, d, page, e4m3, seed=3)
    want = attend(step, fa.Scores(window=window))
    check(step, *want, window=window)
    kp, vp = (x.float() for x in (step.k_pages, step.v_pages))
    for s, (n, m) in enumerate(zip(new, lens)):
        first = m - n - window + 1
        at = first // page
        row = int(step.table_cpu[s, at])
        kp[row, :, :first % page] = float("nan")
        vp[row, :, :first % page] = float("nan")
        step.table_cpu[s, :at] = -5
    step.k_pages.copy_(kp.to(step.k_pages.dtype)), step.v_pages.copy_(vp.to(step.v_pages.dtype))
    step.table.copy_(step.table_cpu)
    for a, b in zip(attend(step, fa.Scores(window=window)), want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("softcap", [0.05, 50.0, 1000.0])
def test_caps(softcap, d, e4m3):
    far = 5.0 if e4m3 else 30.0  # (as far as e4m3 goes)
    for scale, new in ((0.1, [1, 1, 2]), (far, [1, 3, 2]), (far, [100, 3, 1])):
        go(Step(new, [200, 90, 400], 6, 2, d, 64, e4m3, seed=7, k_scale=scale), softcap=softcap)


def test_tokens_past_the_rows_keep_the_others_places():
    """Starts that go on past T: positions, and so distances and windows, are those of the whole
    step, causal or not."""
    import exact_attention_27_gb300 as fa
    d = 64
    for causal in (True, False):
        for new in ([1, 4], [3, 90]):
            step = Step(new, [50, 300], 4, 2, d, 32, seed=2)
            cut = 2
            q = step.q[:step.T - cut]
            scores = fa.Scores(slopes=alibi(4).cuda(), window=40)
            cache, batch = step.handles()
            full = attend(step, scores, causal)
            check(step, *full, slopes=alibi(4), window=40, causal=causal)
            o, lse = fa.paged_attention(cache, batch, q, causal, scores=scores)
            torch.cuda.synchronize()
            assert fa.fa_last_device_error() == 0
            for a, b in zip((o, lse), full):
                err = (a.float() - b[:len(a)].float()).abs().max()
                assert err <= 2 * BF16 * b.float().abs().max()


def test_nothing_to_shape_gives_the_unshaped_bits():
    import exact_attention_27_gb300 as fa
    for new in ([1, 2], [70, 1]):
        step = Step(new, [100, 333], 4, 2, 128, 32, seed=1)
        cache, batch = step.handles()
        a = fa.paged_attention(cache, batch, step.q)
        b = fa.paged_attention(cache, batch, step.q, scores=fa.Scores())
        for x, y in zip(a, b):
            assert torch.equal(x, y)


@pytest.mark.parametrize("new", [[1, 1, 1], [90, 1, 33]])
def test_streams_capture_and_repeat(new):
    """Another stream, and captured steps with their own workspaces replayed at once with other
    lengths, tables and values."""
    import exact_attention_27_gb300 as fa
    d, kw = 128, dict(softcap=20.0, window=200)
    lens = [n + 250 * i + 9 for i, n in enumerate(new)]
    a, b = (Step(new, [m + x for m in lens], 8, 2, d, 16, seed=x, spare=40) for x in (0, 31))
    scores = fa.Scores(**kw)
    one, two = attend(a, scores), attend(a, scores, stream=torch.cuda.Stream())
    for x, y in zip(one, two):
        assert torch.equal(x, y)
    graphs = []
    for step in (a, b):
        cache, batch = step.handles()
        fa.paged_attention(cache, batch, step.q, scores=scores)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            graphs.append((g, fa.paged_attention(cache, batch, step.q, scores=scores)))
    b.kv_lens = [m - 5 for m in b.kv_lens]
    b.k64, b.v64 = ([x[:m] for x, m in zip(y, b.kv_lens)] for y in (b.k64, b.v64))
    b.kv_len.copy_(torch.tensor(b.kv_lens, dtype=torch.int32))
    torch.cuda.synchronize()
    for (g, _), s in zip(graphs, (torch.cuda.Stream(), torch.cuda.Stream())):
        with torch.cuda.stream(s):
            g.replay()
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    for step, (_, out) in zip((a, b), graphs):
        check(step, *out, **kw)


@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_a_layer_of_normed_heads(e4m3):
    """Prompts appended with norms and turn and attended in a window, then single tokens behind
    them, against the dense calls on the same rows."""
    import exact_attention_27_gb300 as fa
    Hq, Hkv, d, page, S = 4, 2, 64, 16, 3
    lens, more = [40, 77, 130], 3
    g = torch.Generator().manual_seed(9)
    total = [n + more for n in lens]
    rows = [torch.randn(n, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda() for n in total]
    norm = fa.HeadNorm((1 + 0.2 * torch.randn(d, generator=g)).cuda(),
                       (1 + 0.2 * torch.randn(d, generator=g)).cuda())
    rotary = fa.Rotary((10000.0 ** (-torch.arange(d // 2) * 2.0 / d)).cuda())
    scores = fa.Scores(softcap=10.0, window=60)
    per = [-(-n // page) for n in total]
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    pages = [torch.full((sum(per), Hkv, page, d), float("nan")).to(dtype).cuda() for _ in range(2)]
    cache = fa.PagedCache(*pages, *((1 / 16, 1 / 16) if e4m3 else (1.0, 1.0)))
    table = torch.full((S, max(per)), -1, dtype=torch.int32)
    order = torch.randperm(sum(per), generator=g).tolist()
    for s in range(S):
        table[s, :per[s]] = torch.tensor(order[sum(per[:s]):sum(per[:s + 1])])
    table = table.cuda()
    got = [[] for _ in range(S)]
    done = [0] * S
    for new in [lens] + [[1] * S] * more:
        x = torch.cat([r[a:a + n] for r, a, n in zip(rows, done, new)])
        done = [a + n for a, n in zip(done, new)]
        starts = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32).cuda()
        batch = fa.PagedBatch(table, starts, torch.tensor(done, dtype=torch.int32).cuda(), max(new))
        q = fa.paged_append(cache, batch, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], rotary, q=x[:, :Hq],
                            norm=norm)
        o, _ = fa.paged_attention(cache, batch, q, scores=scores)
        for s in range(S):
            got[s].append(o[int(starts[s]):int(starts[s + 1])])
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    for s in range(S):
        x = rows[s].transpose(0, 1)[None]
        pos = torch.arange(total[s], dtype=torch.int32, device="cuda")[None]
        q, k = fa.norm_rotary_forward(x[:, :Hq], x[:, Hq:Hq + Hkv], norm, pos, rotary)
        v = x[:, Hq + Hkv:].contiguous()
        o, _ = fa.attention_forward(q, k, v, causal=True, scores=scores)
        err = (torch.cat(got[s]).float() - o[0].transpose(0, 1).float()).norm() / o.float().norm()
        # both round P and o (2^-8 / sqrt 3 each); e4m3 rounds k and v (2^-4 / sqrt 3 each), k's
        # through scores of a standard deviation of about one
        limit = 4 * 2.0 ** -8 / math.sqrt(3) + (2.5 * 2.0 ** -4 / math.sqrt(3) if e4m3 else 0.0)
        assert err <= limit, err
