"""Caps far above and far below the scores, and scores at a cap's ends, against 64-bit values."""

import math

import pytest
import torch

import scores_plain
import test_paged_scores_gpu as paged
from paged_plain import Step
from scores_plain import off_by, whole
from test_scores_gpu import Problem, _built, alibi  # noqa: F401

pytestmark = pytest.mark.gpu


# ------------------------------------------------------------------ caps far above the scores

def share_of_scores(monkeypatch, softcap, far):
    """The bounds' term for the tanh as 2^-21 of the largest score, `far`, in place of the cap: all
    scores lie within 0.4 caps, where the error goes with the score."""
    assert far <= 0.4 * softcap
    monkeypatch.setattr(scores_plain, "TANH", 2.0 ** -21 * far / softcap)


@pytest.mark.parametrize("mode", ["cap", "both"])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("softcap", [3e3, 3e4, 1e5, 1e6, 1e8, 1e15])
def test_caps_far_above_the_scores(monkeypatch, softcap, d, mode):
    p = Problem(1, 2, 1, 200, d, causal=True, softcap=softcap, gain=3.0, seed=d,
                slopes=alibi(2) if mode == "both" else None)
    raw = (p.q.double() @ p.k.double().transpose(2, 3)).abs().max().item() * p.scale
    share_of_scores(monkeypatch, softcap, raw)
    p.check()


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("new", [[1, 2, 1], [100, 3, 40]])
def test_caps_far_above_the_scores_over_pages(monkeypatch, new, d, e4m3):
    """Single tokens and chunks alike: a model's prefill and decode go by one function."""
    for softcap in (3e4, 1e6, 1e8):
        step = Step(new, [200, 90, 400], 6, 2, d, 64, e4m3, seed=7, k_scale=2.0)
        far = step.q_cpu.float().norm(dim=2).max() * max(
            x.norm(dim=2).max() for x in step.k64) / math.sqrt(d)
        share_of_scores(monkeypatch, softcap, far.item())
        paged.go(step, softcap=softcap)


# ------------------------------------------------------------------ caps far below the scores

def derivative_slack(p):
    """What fp32 sums of d products (d + 2 roundings with the scale, 2^-24 of the sum of sizes each)
    do to the cap's derivative: its argument is off by e = (d + 2) 2^-24 size / softcap, and
    1 - tanh^2 moves by 2 tanh (1 - tanh^2) <= 4 / sqrt(27) < 0.77 of that, and by 1 at most.  Heads'
    bounds of dq and dk take this as nothing, which it is but for caps of next to nothing."""
    n, d = p.q.shape[2:]
    dq, dk = torch.zeros(p.q.shape).double(), torch.zeros(p.k.shape).double()
    dist = (torch.arange(n)[:, None] - torch.arange(n)).double()
    for h in range(p.q.shape[1]):
        q, k, v, do = (x.double() for x in (p.q[0, h], p.k[0, 0], p.v[0, 0], p.do[0, h]))
        x = p.softcap * torch.tanh(q @ k.T * p.scale / p.softcap)
        x = x - dist.abs() * (0.0 if p.slopes is None else p.slopes[h].item())
        w = torch.softmax(x.masked_fill(dist < 0, -math.inf), 1)
        dp = do @ v.T
        e = (d + 2) * 2.0 ** -24 * (q.abs() @ k.abs().T) * p.scale / p.softcap
        loose = w * (0.77 * e).clamp(max=1.0) * (dp - (w * dp).sum(1, keepdim=True)).abs()
        dq[0, h] = loose @ k.abs() * p.scale
        dk[0, 0] += loose.T @ q.abs() * p.scale
    return {"dq": dq, "dk": dk}


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("slopes", [None, [0.02, 0.0]])
@pytest.mark.parametrize("gain", [0.005, 0.3])  # within 0.4 caps, and past them
@pytest.mark.parametrize("softcap, scale", [(1e-20, 1e-20), (4e-20, 1e-21), (1e-37, 1e-36),
                                            (1e-15, 1e-15), (1e-8, 0.125), (1e-12, 1e-13)])
def test_caps_whose_square_is_next_to_nothing(softcap, scale, gain, slopes, d):
    """Scores of next to nothing weigh all keys alike; the cap's derivative still tells which
    scores get a gradient."""
    p = Problem(1, 2, 1, 150, d, causal=True, softcap=softcap, scale=scale, slopes=slopes, gain=gain,
                seed=d)
    val, tol = whole(p.q, p.k, p.v, p.see(), scale, softcap, p.slopes, do=p.do)
    for name, x in derivative_slack(p).items():
        tol[name] += x
    got = p.run()
    for name in val:
        assert off_by(got[name], val[name], tol[name]) <= 1, name


# ------------------------------------------------------------------ scores at the ends of a cap

def at_the_end(d, sign, softcap, window, octaves, gain=6.0, N=300):
    """Every score is tanh(sign gain) of the cap; v goes through 2^octaves."""
    p = Problem(1, 2, 1, N, d, causal=True, window=window, softcap=softcap, scale=1.0, seed=d)
    p.q, p.k = torch.zeros_like(p.q), torch.zeros_like(p.k)
    p.q[..., 0], p.k[..., 0] = sign * gain, softcap
    away = torch.tensor([2.0 ** octaves[j % len(octaves)] for j in range(N)])
    p.v = (p.v.float() * away[:, None]).to(torch.bfloat16)
    return p


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("softcap", [30.0, 50.0, 55.0, 56.0])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
def test_a_row_of_one_key_at_the_ends_of_the_cap_is_its_v(d, softcap, sign):
    """To the bit, whatever v's size: v below 2^-40 and beyond 2^40 too."""
    p = at_the_end(d, sign, softcap, 1, range(-40, 41))
    got = p.run()
    assert torch.equal(got["o"].cpu(), p.v.expand(1, 2, 300, d))


@pytest.mark.parametrize("sign", [-1, 1])
@pytest.mark.parametrize("softcap", [50.0, 55.0])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("octave", [-40, -24, -18, -7, 30])
def test_rows_at_the_ends_of_the_cap(octave, d, softcap, sign):
    p = at_the_end(d, sign, softcap, 0, [octave])
    p.do = (p.do.float() * 2.0 ** -octave).to(torch.bfloat16)
    p.check()


# ------------------------------------------------------------------ how far off a capped score is

OFF = 6e-7  # of softcap, and of the score where all lie within 0.4 softcap (include/fa.h)


@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("softcap, scale", [(0.3, 1 / 8), (17.3, 1 / 16), (30.0, 1 / 8),
                                            (50.0, 1 / 8), (55.0, 1.0), (300.0, 1 / 16),
                                            (7e3, 1 / 8), (1e5, 1 / 8), (1e9, 1 / 16)])
def test_capped_scores_are_off_by_as_much_as_stated(softcap, scale, d):
    """Rows of one key, whose lse is the score: q.k is one product, exact in fp32.  With a slope of
    0 the reference is the score itself, so lse adds the roundings of ln 2 and of the product with
    it alone: 2^-23 of the score."""
    import exact_attention_27_gb300 as fa
    N = 4096
    cap, scale = (torch.tensor(x, dtype=torch.float32).item() for x in (softcap, scale))
    worst = [0.0, 0.0]
    for far in (0.39, 12.0):  # all within 0.4 caps, and any
        g = torch.Generator().manual_seed(int(far))
        q = torch.zeros(1, 1, N, d, dtype=torch.bfloat16)
        k = torch.zeros(1, 1, N, d, dtype=torch.bfloat16)
        q[..., 0] = (torch.rand(N, generator=g) * 2 - 1) * far / 1.02
        k[..., 0] = cap / scale * (1 + 0.01 * torch.rand(N, generator=g))
        v = torch.zeros_like(k)
        o, lse = fa.attention_forward(q.cuda(), k.cuda(), v.cuda(), causal=True, scale=scale,
                                      scores=fa.Scores(softcap, torch.zeros(1).cuda(), window=1))
        y = q[..., 0].double() * k[..., 0].double() * scale / cap
        x = cap * torch.tanh(y)
        err = (lse.cpu().double() - x).abs() - 2.0 ** -23 * x.abs()
        if far < 0.4:
            assert y.abs().max() < 0.4
            worst[0] = (err / x.abs().clamp_min(1e-30)).max().item()
        else:
            worst[1] = (err / cap).max().item()
    print(f"softcap {softcap} scale {scale} d {d}: {worst[0]:.2e} {worst[1]:.2e}")
    assert max(worst) <= OFF, worst
