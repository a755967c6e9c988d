"""Shaped scores and head norms on a stream of the caller's, which starts behind what made the
inputs and filled the outputs; gradients where masked keys are large."""

import math

import pytest
import torch

import exact_attention_27_gb300 as fa
from paged_plain import Step
from scores_plain import off_by, whole
from test_paged_scores_gpu import alibi, check
from test_scores_gpu import Problem, _built, i32  # noqa: F401

pytestmark = pytest.mark.gpu


def nan_like(x):
    return torch.full_like(x, float("nan"))


def on(side):
    """`side` behind the current stream's work."""
    side.wait_stream(torch.cuda.current_stream())
    return side


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("kw", [dict(softcap=30.0, window=300), dict(slopes=[0.3, 0.1] * 4)])
def test_both_passes_on_another_stream(d, kw):
    p = Problem(2, 8, 2, 700, d, causal=True, seed=8, **kw)
    want = p.check()
    scores, spans = p.handles()
    q, k, v, do = (x.cuda() for x in (p.q, p.k, p.v, p.do))
    o, dq, dk, dv = nan_like(q), nan_like(q), nan_like(k), nan_like(k)
    lse = torch.full(q.shape[:3], float("nan"), device="cuda")
    ws = fa.scores_workspace(q, k, True)
    ws.fill_(0xFF)
    side = on(torch.cuda.Stream())
    fa.fa_forward_scores(q, k, v, o, lse, p.scale, True, 0, scores, spans, side)
    fa.fa_backward_scores(q, k, v, o, lse, do, dq, dk, dv, p.scale, True, ws, 0, scores, spans, side)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    for name, x in zip(("o", "lse", "dq", "dk", "dv"), (o, lse, dq, dk, dv)):
        assert torch.equal(x, want[name]), name


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[1, 1, 1], [90, 1, 33]])
def test_pages_on_another_stream(new, d, e4m3):
    step = Step(new, [n + 250 * i + 9 for i, n in enumerate(new)], 8, 2, d, 16, e4m3, seed=d)
    kw = dict(softcap=20.0, slopes=alibi(8), window=200)
    scores = fa.Scores(20.0, alibi(8).cuda(), 200)
    cache, batch = step.handles()
    got = []
    for side in (torch.cuda.current_stream(), torch.cuda.Stream()):
        o = nan_like(step.q)
        lse = torch.full((step.T, step.Hq), float("nan"), device="cuda")
        ws = fa.paged_workspace(cache, batch, step.q)
        ws.fill_(0xFF)
        fa.fa_forward_paged(cache, batch, step.q, o, lse, 1 / math.sqrt(d), True, ws, on(side),
                            scores)
        torch.cuda.synchronize()
        assert fa.fa_last_device_error() == 0
        check(step, o, lse, **kw)
        got.append((o, lse))
    for a, b in zip(*got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("softcap", [0.0, 20.0])
def test_gradients_beside_large_masked_keys(d, softcap):
    """Finite keys that no row sees, however large, leave every gradient as it is."""
    N = 200
    p = Problem(1, 2, 1, N, d, end=i32([[150] * N]), softcap=softcap, seed=6)
    val, tol = whole(p.q, p.k, p.v, p.see(), p.scale, softcap, do=p.do)
    p.k[:, :, 150:] = 1e30
    got = p.run()
    for name in val:
        assert off_by(got[name], val[name], tol[name]) <= 1, name
