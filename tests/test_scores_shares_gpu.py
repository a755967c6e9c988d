"""The backward of shaped scores with every number of CTAs that may share a key tile."""

import pytest
import torch

import exact_attention_27_gb300 as fa
from test_scores_gpu import Problem, _built, alibi  # noqa: F401

pytestmark = pytest.mark.gpu

# (B, H_q, H_kv, N_q, N_kv, causal), by head dimension and shares on a GPU of 152 SMs
SHAPES = {
    64: {1: (1, 1, 1, 200, 130, False), 2: (1, 8, 2, 200, 2000, False), 4: (1, 2, 2, 500, 500, True),
         8: (1, 1, 1, 500, 500, True)},
    96: {1: (1, 4, 4, 500, 500, True), 2: (2, 8, 4, 700, 700, True), 4: (1, 4, 2, 200, 300, False),
         8: (1, 2, 1, 200, 130, False)},
    128: {1: (1, 2, 2, 500, 500, True), 2: (2, 16, 4, 200, 300, False), 4: (1, 1, 1, 500, 500, True),
          8: (1, 2, 1, 500, 500, True)},
    256: {1: (1, 1, 1, 500, 500, True), 2: (1, 8, 4, 700, 700, True), 4: (1, 1, 1, 700, 700, True),
          8: (1, 4, 1, 500, 500, True)},
}


def shares(p):
    """What the workspace leaves room for: fp32 sums of dK and dV a share, D and the tiles' spans,
    on 256 bytes each, with 240 to reach the first."""
    (B, Hq, Nq, d), (_, Hkv, Nkv, _) = p.q.shape, p.k.shape

    def up(n):
        return -(-n // 256) * 256
    n = fa.scores_workspace(p.q.cuda(), p.k.cuda(), p.causal).numel()
    n -= up(4 * B * Hq * Nq) + up(8 * B * -(-Nq // 128)) + 240
    each = 2 * 4 * B * Hkv * Nkv * d
    assert n % each == 0
    return n // each or 1


@pytest.mark.parametrize("kw", [{}, dict(softcap=20.0, slopes=True), dict(window=100)])
@pytest.mark.parametrize("n", [1, 2, 4, 8])
@pytest.mark.parametrize("d", list(SHAPES))
def test_shares(d, n, kw):
    if torch.cuda.get_device_properties(0).multi_processor_count != 152:
        pytest.skip("the shapes are for 152 SMs")
    B, Hq, Hkv, Nq, Nkv, causal = SHAPES[d][n]
    kw = dict(kw)
    if kw.pop("slopes", None):
        kw["slopes"] = alibi(Hq)
    p = Problem(B, Hq, Hkv, Nq, d, Nkv=Nkv, causal=causal, seed=d + n, **kw)
    assert shares(p) == n
    a = p.check()
    b = p.run()
    for name in a:
        assert torch.equal(a[name], b[name]), name
