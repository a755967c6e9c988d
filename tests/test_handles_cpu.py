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
