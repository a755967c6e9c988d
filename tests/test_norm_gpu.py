"""Norms of heads' rows with the rotation in the same pass, forward, backward and on the way into a
paged cache, against 64-bit values."""

import pytest
import torch

from norm_plain import backward64, forward64, unit64
from paged_plain import BF16, E4M3, Step, angles64

pytestmark = pytest.mark.gpu
EPS = 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def inv_freq(rot):
    return (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float()


class Problem:
    def __init__(self, B, Hq, Hkv, N, d, rot, interleaved=False, dtype=torch.float32, seed=0,
                 weights=True, gain=2.0):
        g = torch.Generator().manual_seed(seed)
        self.axes = 1 + (d + rot) // 16 % 4
        bf = lambda h: (torch.randn(B, h, N, d, generator=g) * gain).to(torch.bfloat16)  # noqa: E731
        self.q, self.k, self.dq, self.dk = bf(Hq), bf(Hkv), bf(Hq), bf(Hkv)
        self.rot, self.interleaved, self.d = rot, interleaved, d
        self.qw, self.kw = ((1 + 0.3 * torch.randn(d, generator=g)).to(dtype) for _ in range(2))
        if not weights:
            self.qw = self.kw = torch.ones(d)
        self.weights = weights
        if rot:
            self.axis = torch.randint(0, self.axes, (rot // 2,), generator=g)
            self.axis[0] = self.axes - 1
            self.positions = torch.randint(-1000, 10 ** 6, (self.axes, B, N), generator=g).to(
                torch.int32)
            self.inv = inv_freq(rot)
            self.angle = angles64(self.positions, self.inv, self.axis)[:, None]
        else:
            self.angle = None

    def handles(self):
        import exact_attention_27_gb300 as fa
        norm = fa.HeadNorm(self.qw.cuda(), self.kw.cuda(), EPS) if self.weights else \
            fa.HeadNorm(eps=EPS)
        if not self.rot:
            return norm, None, None
        return norm, self.positions.cuda(), fa.Rotary(
            self.inv.cuda(), axis_of_pair=self.axis.tolist(), interleaved=self.interleaved)

    def check_forward(self, q_out, k_out):
        for got, x, w in ((q_out, self.q, self.qw), (k_out, self.k, self.kw)):
            if got is not None:
                want, slack = forward64(x.double(), w.double(), EPS, self.angle, self.rot,
                                        self.interleaved)
                err = (got.cpu().double() - want).abs()
                bound = BF16 * (want.abs() + slack) + slack + 1e-30
                assert torch.all(err <= bound), (err / bound).max().item()

    def check_backward(self, dq, dk, dqw, dkw):
        for dx, dw, x, w, dy in ((dq, dqw, self.q, self.qw, self.dq),
                                 (dk, dkw, self.k, self.kw, self.dk)):
            if dx is None:
                continue
            want, want_w, tol, tol_w = backward64(x.double(), w.double(), EPS, dy.double(),
                                                  self.angle, self.rot, self.interleaved)
            err = (dx.cpu().double() - want).abs()
            assert torch.all(err <= tol), (err / tol).max().item()
            if dw is not None:
                err = (dw.cpu().double() - want_w).abs()
                assert torch.all(err <= tol_w), (err / tol_w).max().item()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 0), (96, 96), (96, 48), (96, 0),
                                   (128, 128), (128, 80), (256, 256), (256, 128), (256, 0)])
@pytest.mark.parametrize("B,Hq,Hkv,N", [(1, 1, 1, 1), (2, 5, 1, 7), (3, 8, 2, 1037),
                                        (1, 32, 32, 40)])
def test_forward_and_backward(B, Hq, Hkv, N, d, rot, interleaved):
    import exact_attention_27_gb300 as fa
    dtype = torch.bfloat16 if (N + d) % 2 else torch.float32
    p = Problem(B, Hq, Hkv, N, d, rot, interleaved, dtype, seed=N + d)
    norm, positions, rotary = p.handles()
    q, k, dq, dk = (x.cuda() for x in (p.q, p.k, p.dq, p.dk))
    p.check_forward(*fa.norm_rotary_forward(q, k, norm, positions, rotary))
    p.check_backward(*fa.norm_rotary_backward(dq, dk, q, k, norm, positions, rotary))
    qo, none = fa.norm_rotary_forward(q, None, norm, positions, rotary)
    assert none is None
    p.check_forward(qo, None)
    out = fa.norm_rotary_backward(dq, None, q, None, norm, positions, rotary)
    assert out[1] is None and out[3] is None
    p.check_backward(out[0], None, out[2], None)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("gain", [1e-6, 1e-3, 300.0])
def test_small_and_large_rows(d, gain):
    """Rows whose mean square lies far below eps, and far above; rows of zeros."""
    import exact_attention_27_gb300 as fa
    p = Problem(1, 3, 2, 50, d, d, gain=gain, weights=gain < 1, seed=d)
    p.q[:, :, 7] = 0
    norm, positions, rotary = p.handles()
    q, k, dq, dk = (x.cuda() for x in (p.q, p.k, p.dq, p.dk))
    p.check_forward(*fa.norm_rotary_forward(q, k, norm, positions, rotary))
    p.check_backward(*fa.norm_rotary_backward(dq, dk, q, k, norm, positions, rotary))


@pytest.mark.parametrize("kind", ["fused", "in place", "broadcast", "over the inputs"])
def test_strides(kind):
    import exact_attention_27_gb300 as fa
    B, Hq, Hkv, N, d = 2, 4, 2, 33, 128
    p = Problem(B, Hq, Hkv, N, d, 64, seed=3)
    norm, positions, rotary = p.handles()
    q, k, dq, dk = (x.cuda() for x in (p.q, p.k, p.dq, p.dk))
    ws = fa.norm_rotary_workspace(d)
    ws.fill_(0xFF)
    dqw, dkw = torch.full((2, d), float("nan"), device="cuda")
    if kind == "fused":  # slices of one projection and of its gradient
        x = torch.cat((q, k), 1).transpose(1, 2).contiguous()
        g = torch.zeros_like(x)
        q2, k2 = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
        p.check_forward(*fa.norm_rotary_forward(q2, k2, norm, positions, rotary))
        fa.fa_norm_rotary_backward(dq, g[:, :, :Hq].transpose(1, 2), dk,
                                   g[:, :, Hq:].transpose(1, 2), q2, k2, norm, dqw, dkw, ws,
                                   positions, rotary)
        p.check_backward(g[:, :, :Hq].transpose(1, 2), g[:, :, Hq:].transpose(1, 2), dqw, dkw)
    elif kind == "in place":
        a, b = q.clone(), k.clone()
        fa.fa_norm_rotary(a, a, b, b, norm, positions, rotary)
        p.check_forward(a, b)
        fa.fa_norm_rotary_backward(dq, dq, dk, dk, q, k, norm, dqw, dkw, ws, positions, rotary)
        p.check_backward(dq, dk, dqw, dkw)
    elif kind == "over the inputs":
        fa.fa_norm_rotary_backward(dq, q, dk, k, q, k, norm, dqw, dkw, ws, positions, rotary)
        p.check_backward(q, k, dqw, dkw)
    else:  # one gradient for all heads
        p.dq = p.dq[:, :1].expand(B, Hq, N, d)
        p.q = p.q[:1].expand(B, Hq, N, d)
        dq, q = p.dq[:, :1].cuda().expand(B, Hq, N, d), p.q[:1].cuda().expand(B, Hq, N, d)
        p.check_forward(*fa.norm_rotary_forward(q, k, norm, positions, rotary))
        p.check_backward(*fa.norm_rotary_backward(dq, dk, q, k, norm, positions, rotary))


def test_weights_not_wanted_and_bits_repeat():
    import exact_attention_27_gb300 as fa
    p = Problem(2, 6, 3, 700, 128, 128, seed=5)
    norm, positions, rotary = p.handles()
    q, k, dq, dk = (x.cuda() for x in (p.q, p.k, p.dq, p.dk))
    ws = fa.norm_rotary_workspace(128)
    a, b = torch.empty_like(q), torch.empty_like(k)
    fa.fa_norm_rotary_backward(dq, a, dk, b, q, k, norm, None, None, ws, positions, rotary)
    p.check_backward(a, b, None, None)
    w = torch.empty(128, device="cuda")
    fa.fa_norm_rotary_backward(dq, a, dk, b, q, k, norm, None, w, ws, positions, rotary)
    p.check_backward(a, b, None, w)
    one = fa.norm_rotary_backward(dq, dk, q, k, norm, positions, rotary)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    two = fa.norm_rotary_backward(dq, dk, q, k, norm, positions, rotary, stream=side)
    torch.cuda.synchronize()
    for x, y in zip(one, two):
        assert torch.equal(x, y)


def test_captured_call_sees_new_values():
    import exact_attention_27_gb300 as fa
    p, p2 = (Problem(1, 4, 2, 90, 64, 64, seed=s) for s in (1, 2))
    norm, positions, rotary = p.handles()
    x = [t.cuda() for t in (p.q, p.k, p.dq, p.dk)]

    def step():
        return (fa.norm_rotary_forward(x[0], x[1], norm, positions, rotary) +
                fa.norm_rotary_backward(x[2], x[3], x[0], x[1], norm, positions, rotary))
    step()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    for t, new in zip(x + [norm.q_weight, norm.k_weight, positions],
                      (p2.q, p2.k, p2.dq, p2.dk, p2.qw, p2.kw, p2.positions)):
        t.copy_(new)
    p2.axis, p2.inv = p.axis, p.inv
    p2.angle = angles64(p2.positions, p.inv, p.axis)[:, None]
    graph.replay()
    torch.cuda.synchronize()
    p2.check_forward(*out[:2])
    p2.check_backward(*out[2:])


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (96, 96), (128, 64), (256, 256), (128, 0)])
@pytest.mark.parametrize("new", [[1, 1, 1], [40, 0, 170, 3]])
def test_append(new, d, rot, e4m3):
    """Rows on their way into the pages: k normed, turned and stored, v as it is, q beside them;
    nothing else of the pages changes, and rows past the last sequence are not written."""
    import exact_attention_27_gb300 as fa
    Hq, Hkv, page = 6, 2, 32
    step = Step(new, [n + 9 * i for i, n in enumerate(new)], Hq, Hkv, d, page, e4m3, seed=d, pad=2)
    cache, batch = step.handles()
    T = step.T
    p = Problem(1, Hq, Hkv, T, d, rot, dtype=torch.bfloat16, seed=7)
    norm, positions, rotary = p.handles()
    rows = lambda x: x[0].transpose(0, 1).contiguous()  # noqa: E731
    q, k = rows(p.q), rows(p.k)
    v = torch.randn(T, Hkv, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    before = [x.view(torch.uint8).clone() for x in (step.k_pages, step.v_pages)]
    out = torch.full((T, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    fa.fa_paged_append(cache, batch, k.cuda(), v.cuda(), rotary,
                       positions[:, 0] if rot else None, q.cuda(), out, norm=norm)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    used = sum(new)
    assert torch.isnan(out[used:]).all()
    angle = None if not rot else p.angle[0, 0][:, None]
    wants = []
    for x, w in ((q, p.qw), (k, p.kw)):
        wants.append(forward64(x.double(), w.double(), EPS, angle, rot))
    want, slack = wants[0]
    err = (out.cpu().double() - want).abs()[:used]
    assert torch.all(err <= (BF16 * (want.abs() + slack) + slack)[:used])
    seen = torch.zeros(step.k_pages.shape[:3], dtype=torch.bool)  # rows stored to
    t = 0
    kp, vp = step.k_pages.cpu().float().double(), step.v_pages.cpu().float().double()
    for s, n in enumerate(new):
        for i in range(n):
            j = step.kv_lens[s] - n + i
            at = (int(step.table_cpu[s, j // page]), slice(None), j % page)
            seen[at] = True
            for pages, x, sl, ds in ((kp, wants[1][0][t + i], wants[1][1][t + i], step.kd),
                                     (vp, v[t + i].double(), torch.zeros(()), step.vd)):
                x = (x / ds).clamp(-448, 448) if e4m3 else x
                sl = sl / ds
                tol = (E4M3 if e4m3 else BF16) * (x.abs() + sl) + sl + (2.0 ** -10 if e4m3 else 0)
                assert torch.all((pages[at] - x).abs() <= tol)
        t += n
    for pages, old in zip((step.k_pages, step.v_pages), before):
        assert torch.equal(pages.view(torch.uint8).cpu()[~seen], old.cpu()[~seen])


def test_norm_then_shaped_attention_then_back():
    """A layer's part of a training step: norms and turn, attention with capped scores over packed
    documents, and the way back to q, k, v and both weights, against 64-bit autograd."""
    import math

    import exact_attention_27_gb300 as fa
    B, Hq, Hkv, N, d = 2, 4, 2, 190, 64
    p = Problem(B, Hq, Hkv, N, d, d, seed=11)
    g = torch.Generator().manual_seed(4)
    v, do = (torch.randn(B, h, N, d, generator=g).to(torch.bfloat16) for h in (Hkv, Hq))
    norm, positions, rotary = p.handles()
    scores = fa.Scores(softcap=8.0)
    bounds = torch.tensor([[0, 60, 61, 180], [0, 100, 150, 190]], dtype=torch.int32)
    spans = fa.KeySpans.documents(bounds.cuda(), N)
    kw = dict(causal=True, scores=scores, spans=spans)
    qn, kn = fa.norm_rotary_forward(p.q.cuda(), p.k.cuda(), norm, positions, rotary)
    o, lse = fa.attention_forward(qn, kn, v.cuda(), **kw)
    dq, dk, dv = fa.attention_backward(qn, kn, v.cuda(), o, lse, do.cuda(), **kw)
    dq, dk, dqw, dkw = fa.norm_rotary_backward(dq, dk, p.q.cuda(), p.k.cuda(), norm, positions,
                                               rotary)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0

    leaves = [x.double().requires_grad_() for x in (p.q, p.k, v, p.qw, p.kw)]
    phase = torch.polar(torch.ones_like(p.angle), p.angle)

    def turned(x, w):
        x = unit64(x, EPS)[0] * w
        z = torch.complex(x[..., :d // 2], x[..., d // 2:]) * phase
        return torch.cat((z.real, z.imag), -1)
    q64, k64 = turned(leaves[0], leaves[3]), turned(leaves[1], leaves[4])
    k64, v64 = (x.repeat_interleave(Hq // Hkv, 1) for x in (k64, leaves[2]))
    s = 8 * torch.tanh(q64 @ k64.transpose(2, 3) / math.sqrt(d) / 8)
    row = torch.arange(N)
    doc = torch.stack([torch.searchsorted(b, row.int(), right=True) for b in bounds])
    see = (doc[:, :, None] == doc[:, None]) & (row[:, None] >= row) & (doc < 4)[:, :, None]
    live = see.any(-1)[:, None, :, None]
    w = torch.softmax(s.masked_fill(~see[:, None], -1e300), -1) * live
    grads = torch.autograd.grad(w @ v64, leaves, do.double())
    # Relative to each tensor's norm: the roundings of q, k, P, dS, o, dq and dk to bf16 (half
    # steps of 2^-8, spread evenly: 2^-8 / sqrt(3) each), seven of them in a row at most, each
    # scaled by what is downstream of it (scores of a standard deviation of 2 to 4: a rounding of
    # q moves P by up to 4 x 2^-8 of itself)
    limit = (3 + 4 * 4) * 2.0 ** -8 / math.sqrt(3)
    for got, want in zip((dq, dk, dv, dqw, dkw), grads):
        err = (got.cpu().double() - want).norm() / want.norm()
        assert err <= limit, err


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("B,N", [(2, 1901), (900, 5), (1, 7407), (3, 4999)])
def test_many_positions(B, N, d):
    """Blocks of several positions, and of the gradient's kernel several steps each, some of them
    over many short batch entries."""
    import exact_attention_27_gb300 as fa
    p = Problem(B, 3, 1, N, d, d if N % 2 else d // 2, interleaved=B == 1, seed=N)
    norm, positions, rotary = p.handles()
    q, k, dq, dk = (x.cuda() for x in (p.q, p.k, p.dq, p.dk))
    p.check_forward(*fa.norm_rotary_forward(q, k, norm, positions, rotary))
    p.check_backward(*fa.norm_rotary_backward(dq, dk, q, k, norm, positions, rotary))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("new", [[2, 1500, 1, 900, 1600], [7400, 3], [1] * 40, [9000, 6000]])
@pytest.mark.parametrize("with_q", [True, False])
def test_append_many_rows_at_their_places(new, d, e4m3, with_q):
    """Steps of many tokens and of many sequences, positions those in the sequences, with and
    without q."""
    import exact_attention_27_gb300 as fa
    Hq, Hkv, page = 3, 1, 64
    past = [(5 * i) % 23 for i in range(len(new))]
    step = Step(new, [n + m for n, m in zip(new, past)], Hq, Hkv, d, page, e4m3, seed=d)
    cache, batch = step.handles()
    T = step.T
    place = torch.cat([torch.arange(m, m + n) for n, m in zip(new, past)])
    p = Problem(1, Hq, Hkv, T, d, d, dtype=torch.bfloat16, seed=T)
    p.axes, p.axis = 1, torch.zeros(d // 2, dtype=torch.long)
    p.angle = angles64(place.to(torch.int32)[None, None], p.inv, p.axis)[:, None]
    norm, _, rotary = p.handles()
    rows = lambda x: x[0].transpose(0, 1).contiguous().cuda()  # noqa: E731
    v = torch.randn(T, Hkv, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16)
    out = torch.full((T, Hq, d), float("nan"), dtype=torch.bfloat16, device="cuda")
    fa.fa_paged_append(cache, batch, rows(p.k), v.cuda(), rotary, None,
                       rows(p.q) if with_q else None, out if with_q else None, norm=norm)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    if with_q:
        p.check_forward(out.transpose(0, 1)[None], None)
    seq = torch.cat([torch.full((n,), s) for s, n in enumerate(new)])
    where = step.table_cpu[seq, place // page].long(), place % page
    want, slack = forward64(p.k.double(), p.kw.double(), EPS, p.angle, d)
    for pages, x, sl, ds in ((step.k_pages, want[0].transpose(0, 1), slack[0].transpose(0, 1),
                              step.kd),
                             (step.v_pages, v.double(), torch.zeros(()), step.vd)):
        got = pages.cpu().float().double()[where[0], :, where[1]]
        x = (x / ds).clamp(-448, 448) if e4m3 else x
        sl = sl / ds
        tol = (E4M3 if e4m3 else BF16) * (x.abs() + sl) + sl + (2.0 ** -10 if e4m3 else 0)
        assert torch.all((got - x).abs() <= tol)


def test_offsets_past_32_bits():
    """Positions so far apart in memory that their offsets pass 2^31 values."""
    import exact_attention_27_gb300 as fa
    B, H, N, d = 1, 3, 21, 128
    p = Problem(B, H, H, N, d, d, seed=9)
    norm, positions, rotary = p.handles()
    q, k, dq, dk = (x.cuda() for x in (p.q, p.k, p.dq, p.dk))
    apart = 2 ** 31 // 20 // 64 * 64 + 64
    far = [torch.empty(20 * apart + H * d, dtype=torch.bfloat16, device="cuda") for _ in range(3)]
    x, g, out = (t.as_strided((B, H, N, d), (0, d, apart, 1)) for t in far)
    x.copy_(q)
    g.copy_(dq)
    a, b = torch.empty_like(q), torch.empty_like(k)
    fa.fa_norm_rotary(x, out, k, b, norm, positions, rotary)
    p.check_forward(out, b)
    dqw, dkw = torch.empty(2, d, device="cuda")
    ws = fa.norm_rotary_workspace(d)
    fa.fa_norm_rotary_backward(g, out, dk, b, x, k, norm, dqw, dkw, ws, positions, rotary)
    p.check_backward(out, b, dqw, dkw)
    fa.fa_norm_rotary_backward(g, a, None, None, x, None, norm, None, None, ws, positions, rotary)
    assert torch.equal(a, out)
