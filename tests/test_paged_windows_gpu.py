"""Windows over a paged cache for tokens that lie before their sequence, near and far."""

import pytest
import torch

import exact_attention_27_gb300 as fa
from paged_plain import Step
from test_paged_scores_gpu import attend, check
from test_scores_gpu import _built  # noqa: F401

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("window", [1, 7, 2 ** 31 - 30, 2 ** 31 - 1])
@pytest.mark.parametrize("new, lens", [([6, 2], [4, 30]), ([40, 3, 150], [20, 30, 60])])
def test_more_new_tokens_than_positions(new, lens, window, causal, d, e4m3):
    """A length below a sequence's new tokens: the first of them lie before position 0, beside others
    that see keys.  A window past all positions leaves everything in."""
    step = Step(new, lens, 4, 2, d, 16, e4m3, seed=d)
    check(step, *attend(step, fa.Scores(window=window), causal), window=window, causal=causal)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("rows", [2, 90])
@pytest.mark.parametrize("end", [1000, 2 ** 31 - 1])
def test_starts_far_past_the_rows(end, rows, d, e4m3):
    """The last start lies far past the step's rows, so that those lie far before the sequence; not
    causal, they see all of it."""
    step = Step([1, rows], [50, 77], 4, 2, d, 16, e4m3, seed=d)
    step.q_start[-1] = end
    check(step, *attend(step, fa.Scores(window=100), False), causal=False)
    o, lse = attend(step, fa.Scores(window=100), True)
    assert not torch.any(o[1:]) and torch.all(lse[1:] == -torch.inf)
