"""Attention with shaped scores, forward and backward, against 64-bit values."""

import math

import pytest
import torch

from scores_plain import off_by, spans_of, whole

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


class Problem:
    """Inputs from a seed, the library's call into NaN outputs, and the check of what it gives."""

    def __init__(self, B, Hq, Hkv, Nq, d, Nkv=None, softcap=0.0, slopes=None, window=0, causal=False,
                 q_offset=0, first=None, end=None, gain=2.0, seed=0, scale=None):
        g = torch.Generator().manual_seed(seed)
        Nkv = Nkv or Nq
        bf = lambda *s: torch.randn(s, generator=g).to(torch.bfloat16)  # noqa: E731
        self.q = (bf(B, Hq, Nq, d).float() * gain).to(torch.bfloat16)
        self.k, self.v, self.do = bf(B, Hkv, Nkv, d), bf(B, Hkv, Nkv, d), bf(B, Hq, Nq, d)
        self.scale = scale or 1.0 / math.sqrt(d)
        self.softcap, self.window, self.causal, self.q_offset = softcap, window, causal, q_offset
        self.slopes = None if slopes is None else torch.tensor(slopes, dtype=torch.float32)
        # spans as [B or 1, Nq] int32, or None
        self.first, self.end = first, end

    def see(self):
        def row(x, b):
            return None if x is None else x[b % x.shape[0]]
        return [spans_of(self.q.shape[2], self.k.shape[2], self.causal, self.q_offset, self.window,
                         row(self.first, b), row(self.end, b)) for b in range(self.q.shape[0])]

    def handles(self):
        import exact_attention_27_gb300 as fa
        slopes = None if self.slopes is None else self.slopes.cuda()
        scores = fa.Scores(self.softcap, slopes, self.window)
        spans = None
        if self.first is not None or self.end is not None:
            spans = fa.KeySpans(*(None if x is None else x.cuda() for x in (self.first, self.end)))
        return scores, spans

    def run(self, stream=None):
        import exact_attention_27_gb300 as fa
        scores, spans = self.handles()
        q, k, v, do = (x.cuda() for x in (self.q, self.k, self.v, self.do))
        nan = [torch.full_like(x, float("nan")) for x in (q, q, k, k)]
        o, dq, dk, dv = nan
        lse = torch.full(q.shape[:3], float("nan"), device="cuda")
        fa.fa_forward_scores(q, k, v, o, lse, self.scale, self.causal, self.q_offset, scores, spans,
                             stream)
        ws = fa.scores_workspace(q, k, self.causal, self.q_offset)
        ws.fill_(0xFF)
        if stream is not None:
            stream.wait_stream(torch.cuda.current_stream())
        fa.fa_backward_scores(q, k, v, o, lse, do, dq, dk, dv, self.scale, self.causal, ws,
                              self.q_offset, scores, spans, stream)
        torch.cuda.synchronize()
        assert fa.fa_last_device_error() == 0
        return {"o": o, "lse": lse, "dq": dq, "dk": dk, "dv": dv}

    def check(self, got=None):
        got = got or self.run()
        val, tol = whole(self.q, self.k, self.v, self.see(), self.scale, self.softcap, self.slopes,
                         self.q_offset, self.do)
        for name in val:
            x = off_by(got[name], val[name], tol[name])
            assert x <= 1, f"{name} off by {x:.2f} of its bound"
        return got


def alibi(H):
    return [2.0 ** (-8.0 * (h + 1) / H) for h in range(H)]


def i32(x):
    return torch.as_tensor(x, dtype=torch.int32)


def documents(N, lengths):
    first, end = [], []
    for n in lengths:
        a = len(first)
        first += [a] * n
        end += [a + n] * n
    pad = N - len(first)
    return first + [0] * pad, end + [0] * pad


MODES = {"plain": {}, "slopes": {"slopes": True}, "cap": {"softcap": 20.0},
         "both": {"softcap": 20.0, "slopes": True}, "high": {"softcap": 70.0}}


def masks(N, kind):
    if kind == "documents":  # two packings; the ends of both are padding
        a, b = documents(N, [1, 70, 2, 60, N - 150]), documents(N, [N // 2, 1, 1])
        return {"causal": True, "first": i32([a[0], b[0]]), "end": i32([a[1], b[1]])}
    if kind == "two-sided":  # documents seen both ways
        a, b = documents(N, [30, N - 60]), documents(N, [N])
        return {"first": i32([a[0], b[0]]), "end": i32([a[1], b[1]])}
    if kind == "prefix":
        return {"end": i32([[max(i + 1, p) for i in range(N)] for p in (N // 3, 1)])}
    if kind == "padded":
        return {"end": i32([[N - 40] * N, [7] * N])}
    if kind == "window":
        return {"causal": True, "window": 50}
    if kind == "window both ways":  # a window bounds what lies behind; ahead all is seen
        return {"window": 20}
    if kind == "anything":  # any spans, empty ones among them, beyond both ends too
        g = torch.Generator().manual_seed(N)
        first = torch.randint(-20, N, (2, N), generator=g)
        return {"first": i32(first), "end": i32(first + torch.randint(-5, N, (2, N), generator=g))}
    return {"causal": kind == "causal"}


@pytest.mark.parametrize("mode", list(MODES))
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("kind", ["causal", "full", "documents", "two-sided", "prefix", "padded",
                                  "window", "window both ways", "anything"])
def test_masks(kind, d, mode):
    N = 300
    kw = dict(MODES[mode])
    if kw.pop("slopes", None):
        kw["slopes"] = alibi(4)
    Problem(2, 4, 2, N, d, seed=d + len(kind), **masks(N, kind), **kw).check()


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("N", [1, 2, 3, 63, 64, 65, 127, 128, 129, 257, 385, 513])
def test_lengths(N, d):
    Problem(1, 3, 1, N, d, causal=True, softcap=50.0, slopes=alibi(3), seed=N).check()


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("sizes", [(1, 500, 499, 0), (130, 700, 570, 0), (5, 9, 4, 3),
                                   (200, 60, 0, 0), (129, 300, 1000, 40), (64, 64, 40, 0)])
def test_queries_behind_a_history(sizes, d):
    """N_q and N_kv apart, positions past the keys, windows that end before any key."""
    Nq, Nkv, off, window = sizes
    Problem(2, 4, 4, Nq, d, Nkv=Nkv, q_offset=off, causal=True, window=window, softcap=30.0,
            seed=Nq).check()
    Problem(2, 4, 4, Nq, d, Nkv=Nkv, q_offset=off, slopes=[0.5, 0.01, -0.02, 0.0],
            seed=Nq).check()


@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("softcap", [0.01, 1.0, 30.0, 55.0, 56.0, 300.0, 1e6])
def test_caps(softcap, d):
    """Scores far below, around and far past the cap; caps on both sides of the fixed
    reference."""
    for gain in (0.05, 3.0, 40.0):
        Problem(1, 2, 1, 200, d, causal=True, softcap=softcap, gain=gain, seed=3).check()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_some_rows_past_the_tanh_polynomial(d):
    """One row in a warp past it takes the whole warp the other way."""
    p = Problem(1, 2, 2, 256, d, softcap=20.0, seed=5)
    p.q[:, :, 40] *= 30
    p.q[:, :, 200] *= 8
    p.check()


@pytest.mark.parametrize("d", [64, 128, 256])
def test_steep_and_rising_slopes(d):
    """Weights that fall by 2^-30 a step, and that rise with the distance."""
    Problem(1, 3, 1, 300, d, causal=True, slopes=[20.0, -0.3, 1000.0], seed=9).check()


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_far_positions(d):
    """Distances past 2^24, where fp32 no longer holds every whole number."""
    Problem(1, 2, 1, 140, d, Nkv=150, q_offset=2 ** 25 + 3, causal=True, slopes=[1e-7, 1e-6],
            seed=2).check()


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_nothing_seen_at_all(d):
    got = Problem(1, 2, 1, 130, d, end=i32([[0] * 130]), softcap=5.0).check()
    for name in ("o", "dq", "dk", "dv"):
        assert torch.all(got[name] == 0)


@pytest.mark.parametrize("d", [64, 256])
def test_one_key_a_row_has_no_score_gradient(d):
    got = Problem(1, 2, 1, 300, d, causal=True, window=1, softcap=5.0).check()
    assert torch.all(got["dq"] == 0) and torch.all(got["dk"] == 0)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_long(d):
    N = 2500
    a = documents(N, [900, 3, 1200, 300])
    Problem(1, 2, 1, N, d, causal=True, first=i32([a[0]]), end=i32([a[1]]), softcap=50.0,
            seed=d).check()
    Problem(1, 2, 2, N, d, causal=True, window=700, slopes=alibi(2), seed=d + 1).check()


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_agrees_with_the_unshaped_calls(d):
    """Without anything to shape, fa_forward's and fa_backward's values."""
    import exact_attention_27_gb300 as fa
    p = Problem(2, 4, 2, 333, d, causal=True, seed=1)
    got = p.check()
    q, k, v, do = (x.cuda() for x in (p.q, p.k, p.v, p.do))
    o, lse = fa.attention_forward(q, k, v, causal=True)
    grads = fa.attention_backward(q, k, v, o, lse, do, causal=True)
    val, tol = whole(p.q, p.k, p.v, p.see(), p.scale, do=p.do)
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + tuple(grads)):
        assert off_by(x, val[name], tol[name]) <= 1
        assert ((got[name] - x).abs().double().cpu() <= 2 * tol[name]).all()


def test_one_row_of_spans_for_all_and_spans_in_wider_tensors():
    import exact_attention_27_gb300 as fa
    N, d = 200, 64
    first, end = (i32([x]) for x in documents(N, [50, 100, 30]))
    p = Problem(3, 2, 1, N, d, causal=True, first=first, end=end, seed=4)
    ref = p.check()
    q, k, v, do = (x.cuda() for x in (p.q, p.k, p.v, p.do))
    wide = torch.full((3, 2, N + 24), -9, dtype=torch.int32, device="cuda")
    wide[:, 0, :N], wide[:, 1, :N] = first.cuda(), end.cuda()
    for spans in (fa.KeySpans(first[0].cuda(), end[0].cuda()),
                  fa.KeySpans(wide[:, 0, :N], wide[:, 1, :N])):
        o, lse = fa.attention_forward(q, k, v, causal=True, spans=spans)
        grads = fa.attention_backward(q, k, v, o, lse, do, causal=True, spans=spans)
        for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse) + tuple(grads)):
            assert torch.equal(ref[name], x), name


def test_span_helpers():
    import exact_attention_27_gb300 as fa
    N = 20
    bounds = i32([[0, 5, 5, 12, 18], [2, 3, 4, 5, 20]]).cuda()
    s = fa.KeySpans.documents(bounds, N)
    assert s.first[0].tolist() == [0] * 5 + [5] * 7 + [12] * 6 + [0] * 2
    assert s.end[0].tolist() == [5] * 5 + [12] * 7 + [18] * 6 + [0] * 2
    assert s.first[1].tolist() == [0, 0, 2, 3, 4] + [5] * 15
    assert s.end[1].tolist() == [0, 0, 3, 4, 5] + [20] * 15
    one = fa.KeySpans.documents(bounds[0], N)
    assert one.first.tolist() == s.first[0].tolist() and one.B == 1
    p = fa.KeySpans.prefix(i32([3, 0]).cuda(), 4, q_offset=1)
    assert p.end.tolist() == [[3, 3, 4, 5], [2, 3, 4, 5]]
    assert fa.KeySpans.lengths(i32([3, 9]).cuda(), 2).end.tolist() == [[3, 3], [9, 9]]


@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_bits_repeat_and_another_stream(d):
    p = Problem(2, 8, 2, 700, d, causal=True, softcap=30.0, window=300, seed=8)
    a, b = p.run(), p.run()
    side = torch.cuda.Stream()
    c = p.run(side)
    for name in a:
        assert torch.equal(a[name], b[name]) and torch.equal(a[name], c[name]), name


def test_captured_steps_see_new_spans():
    """A captured training step replays with the spans and values that its tensors then hold; two
    captured steps may replay at once."""
    import exact_attention_27_gb300 as fa
    B, H, N, d = 1, 4, 260, 64
    probs = [Problem(B, H, 2, N, d, causal=True, softcap=20.0, seed=s,
                     first=i32([documents(N, ls)[0]]), end=i32([documents(N, ls)[1]]))
             for s, ls in enumerate(([100, 160], [1, 200, 40], [260]))]
    steps = []
    for _ in range(2):
        x = [t.cuda() for t in (probs[0].q, probs[0].k, probs[0].v, probs[0].do, probs[0].first,
                                probs[0].end)]
        scores, spans = fa.Scores(20.0), fa.KeySpans(x[4], x[5])

        def step(x=x, scores=scores, spans=spans):
            o, lse = fa.attention_forward(*x[:3], causal=True, scores=scores, spans=spans)
            return (o, lse) + fa.attention_backward(*x[:3], o, lse, x[3], causal=True,
                                                    scores=scores, spans=spans)
        step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = step()
        steps.append((x, graph, out))
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for pair in ((1, 2), (2, 0)):
        for (x, _, _), i in zip(steps, pair):
            p = probs[i]
            for t, new in zip(x, (p.q, p.k, p.v, p.do, p.first, p.end)):
                t.copy_(new)
        torch.cuda.synchronize()
        for s, (_, graph, _) in zip(streams, steps):
            with torch.cuda.stream(s):
                graph.replay()
        torch.cuda.synchronize()
        assert fa.fa_last_device_error() == 0
        for (_, _, out), i in zip(steps, pair):
            probs[i].check(dict(zip(("o", "lse", "dq", "dk", "dv"), out)))


@pytest.mark.parametrize("d", [64, 128, 256])
def test_masked_keys_may_hold_anything(d):
    """Scores of keys that no row sees never count, whatever k holds there (v must be finite): the
    values and bounds are those of the finite k.  (Not the bits: of the two ways to a tanh, each
    within 2e-7, a warp takes the one that all of its scores allow, masked ones among them.)"""
    N = 200
    p = Problem(1, 2, 1, N, d, end=i32([[150] * N]), softcap=20.0, seed=6)
    k = p.k.clone()
    for far in (float("inf"), float("nan"), 1e30):
        p.k[:, :, 150:] = far
        got = p.run()
        p.k = k.clone()
        if not math.isfinite(far):  # dk of such keys is 0, and dq never takes them in
            got["dq"] = None
        val, tol = whole(p.q, p.k, p.v, p.see(), p.scale, p.softcap, do=p.do)
        for name in ("o", "lse", "dv", "dk"):
            assert off_by(got[name], val[name], tol[name]) <= 1, name


@pytest.mark.parametrize("softcap", [0.0, 30.0])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_long_windows_and_steep_heads(d, softcap):
    """Windows past the keys that dQ goes through twice, with a history and without; heads whose
    few keys that count lie among many; distances of both signs over long rows."""
    N = 2300
    Problem(1, 3, 1, N, d, causal=True, window=1500, softcap=softcap, seed=d).check()
    Problem(1, 2, 1, N, d, Nkv=N + 700, q_offset=700, causal=True, window=1000, softcap=softcap,
            seed=d + 1).check()
    Problem(1, 3, 3, N, d, causal=True, softcap=softcap, slopes=[0.7, 0.12, 0.05],
            seed=d + 2).check()
    Problem(1, 2, 1, 1400, d, softcap=softcap, slopes=[-0.2, 0.1], q_offset=90, seed=d + 3).check()


def test_offsets_past_32_bits():
    """More than 2^31 values of k: 5 queries at its end, behind a window."""
    import exact_attention_27_gb300 as fa
    d, few, many = 128, 1100, 17_000_000
    p = Problem(1, 2, 1, 5, d, Nkv=few, q_offset=few - 5, causal=True, window=1000,
                slopes=[0.3, 0.01], seed=4)
    scores, _ = p.handles()
    q, do = p.q.cuda(), p.do.cuda()
    k, v = (torch.zeros(1, 1, many, d, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    k[:, :, -few:], v[:, :, -few:] = p.k.cuda(), p.v.cuda()
    o, lse = fa.attention_forward(q, k, v, causal=True, q_offset=many - 5, scores=scores)
    dq, dk, dv = fa.attention_backward(q, k, v, o, lse, do, causal=True, q_offset=many - 5,
                                       scores=scores)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    assert not torch.any(dk[:, :, :-few]) and not torch.any(dv[:, :, :-few])
    p.check({"o": o, "lse": lse, "dq": dq, "dk": dk[:, :, -few:], "dv": dv[:, :, -few:]})


@pytest.mark.parametrize("softcap", [0.0, 5.0, 50.0, 70.0])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_a_row_of_one_key_is_its_v(d, softcap):
    """To the bit: v is in bf16, and the weight over itself is 1 to fp32."""
    p = Problem(1, 2, 1, 300, d, causal=True, window=1, softcap=softcap, seed=d)
    got = p.run()
    assert torch.equal(got["o"].cpu(), p.v.expand(1, 2, 300, d))
    p.check(got)
