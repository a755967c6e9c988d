"""Handles and calls refuse what they would otherwise take for something else."""

import pytest
import torch

import exact_attention_27_gb300 as fa
from exact_attention_27_gb300 import paged


def test_a_norm_on_cuda_is_on_the_current_device(monkeypatch):
    paged._load_torch()
    monkeypatch.setattr(paged, "_device", lambda: 1)
    assert fa.HeadNorm(device="cuda").device == 1
    assert fa.HeadNorm().device == 1
    assert fa.HeadNorm(device="cuda:0").device == 0
    assert fa.HeadNorm(device=torch.device("cuda", 2)).device == 2


def test_a_norm_is_on_a_gpu():
    with pytest.raises(ValueError):
        fa.HeadNorm(device="cpu")


@pytest.mark.parametrize("softcap", [1e-50, 1e39, -1e-50])
def test_a_cap_that_fp32_does_not_hold_is_refused(softcap):
    """1e-50 would be no cap at all."""
    with pytest.raises(ValueError):
        fa.Scores(softcap)


@pytest.mark.parametrize("q_offset", [2 ** 32, 2 ** 32 + 40, 2 ** 31, -2 ** 31 - 1])
def test_offsets_past_32_bits_are_refused(q_offset):
    """2^32 would be 0."""
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    lse = torch.zeros(1, 2, 8)
    calls = [lambda: fa.fa_forward_ex(x, x, x, x, lse, 0.1, True, q_offset),
             lambda: fa.fa_forward_scores(x, x, x, x, lse, 0.1, True, q_offset),
             lambda: fa.fa_backward_scores(x, x, x, x, lse, x, x, x, x, 0.1, True, x, q_offset),
             lambda: fa.scores_workspace(x, x, True, q_offset),
             lambda: fa.attention_forward(x, x, x, True, q_offset=q_offset, scores=fa.Scores(9.0)),
             lambda: fa.attention_backward(x, x, x, x, lse, x, True, q_offset=q_offset)]
    for call in calls:
        with pytest.raises(ValueError, match="q_offset"):
            call()
