"""Caps far above the scores, against 64-bit values."""

import math

import pytest
import torch

import scores_plain
import test_paged_scores_gpu as paged
from paged_plain import Step
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
