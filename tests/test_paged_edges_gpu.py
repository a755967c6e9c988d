"""Calls at the edges of what the paged and rotary entry points take."""

import math

import pytest
import torch

from paged_plain import Step, attention64, attention_bounds

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("d", [64, 256])
@pytest.mark.parametrize("cut", [9, 2, 60])
def test_starts_past_the_last_row(cut, d, causal, e4m3):
    """A step whose starts go on past its T rows (a batch used again with fewer rows): the tokens
    that have rows keep their places, in the append and in the attention; the others are neither
    stored nor answered.  `cut` rows are missing: of one sequence, of a short draft, of more than
    a whole sequence."""
    import exact_attention_27_gb300 as fa
    new = [3, 2, 4] if cut == 2 else [3, 40, 12, 30]
    total = [50, 90, 9] if cut == 2 else [50, 90, 60, 31]
    step = Step(new, total, 4, 2, d, 16, e4m3, seed=cut + d)
    cache, batch = step.handles()
    T = step.T - cut
    q = step.q[:T]
    before = [x.clone() for x in (step.k_pages, step.v_pages)]
    # the rows that the pages hold already: what is stored again must land in its own place
    old = [torch.cat([x[m - n:m] for x, n, m in zip(xs, new, total)])[:T]
           for xs in (step.k64, step.v64)]
    k, v = (x.to(torch.bfloat16).cuda() for x in old)
    inv = torch.zeros(8, device="cuda")  # (turns nothing)
    q_out = fa.paged_append(cache, batch, k, v, fa.Rotary(inv), q=q)
    o, lse = fa.paged_attention(cache, batch, q, causal)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    assert torch.equal(q_out, q)
    for now, was in zip((step.k_pages, step.v_pages), before):
        assert torch.equal(now.view(torch.uint8), was.view(torch.uint8))
    at = 0
    for s, (n, m) in enumerate(zip(new, total)):
        rows = min(n, T - at)
        if rows <= 0:
            break
        ro, rl, a, size = attention64(step.q_cpu[at:at + rows].double(), step.k64[s], step.v64[s],
                                      1 / math.sqrt(d), causal, m - n)
        ot, lt = attention_bounds(ro, rl, a, size, d, m, step.v64[s].abs().max().item(), e4m3)
        assert torch.all((o[at:at + rows].cpu().double() - ro).abs() <= ot), s
        assert torch.all((lse[at:at + rows].cpu().double() - rl).abs() <= lt), s
        at += n


@pytest.mark.parametrize("fn", ["fa_rotary", "fa_rotary_backward"])
def test_k_without_its_output_is_refused(fn):
    """One of k and k_out alone: an output that nothing would write, or a tensor to turn into
    nothing."""
    import exact_attention_27_gb300 as fa
    x = torch.randn(1, 2, 8, 64, device="cuda").to(torch.bfloat16)
    y, z = torch.empty_like(x), torch.empty_like(x)
    positions = torch.arange(8, dtype=torch.int32, device="cuda")[None]
    rotary = fa.Rotary(torch.ones(32, device="cuda"))
    for k, k_out in ((x, None), (None, z)):
        with pytest.raises(ValueError, match="neither"):
            getattr(fa, fn)(x, y, k, k_out, positions, rotary)
    getattr(fa, fn)(x, y, None, None, positions, rotary)
    getattr(fa, fn)(x, y, x, z, positions, rotary)
    torch.cuda.synchronize()
    assert torch.equal(y, z)
