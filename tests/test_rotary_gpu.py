"""Rotary positions with several axes, forward and backward, against 64-bit values."""

import math

import pytest
import torch

from paged_plain import BF16, angles64, turn64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def inv_freq(rot):
    return (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float()


def check(got, x, positions, inv, axis, rot, interleaved, sign=1.0):
    """x [B, H, N, d] on the CPU, positions [axes, B, N]."""
    angle = sign * angles64(positions, inv, axis)[:, None]
    want, slack = turn64(x.double(), angle, rot, interleaved)
    err = (got.cpu().double() - want).abs()
    bound = BF16 * want.abs() + slack
    assert torch.all(err <= bound), (err / bound.clamp(min=1e-30)).max().item()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (96, 96), (96, 48), (128, 128), (128, 80),
                                   (256, 256), (256, 128)])
@pytest.mark.parametrize("B,Hq,Hkv,N", [(1, 1, 1, 1), (2, 5, 1, 7), (3, 8, 2, 1037)])
def test_forward_and_backward(B, Hq, Hkv, N, d, rot, interleaved):
    import exact_attention_27_gb300 as fa
    g = torch.Generator().manual_seed(N + d)
    axes = 1 + (d + rot) // 16 % 4
    q, k = (torch.randn(B, h, N, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv))
    axis = torch.randint(0, axes, (rot // 2,), generator=g)
    axis[0] = axes - 1
    positions = torch.randint(-1000, 10 ** 6, (axes, B, N), generator=g).to(torch.int32)
    inv = inv_freq(rot)
    rotary = fa.Rotary(inv.cuda(), axis_of_pair=axis.tolist(), interleaved=interleaved)
    args = (q.cuda(), k.cuda(), positions.cuda(), rotary)
    for go, sign in ((fa.rotary_forward, 1.0), (fa.rotary_backward, -1.0)):
        qo, ko = go(*args)
        torch.cuda.synchronize()
        check(qo, q, positions, inv, axis, rot, interleaved, sign)
        check(ko, k, positions, inv, axis, rot, interleaved, sign)
    qo, none = fa.rotary_forward(q.cuda(), None, positions.cuda(), rotary)
    assert none is None
    check(qo, q, positions, inv, axis, rot, interleaved)


def test_far_positions():
    """Positions up to 2^31: only the turn's fraction counts, and fp32 angles would lose it.  The
    fraction of f / 2 pi is kept to 2^-53 of itself, so at 2^31 and f = 1 the angle is off by
    2^31 x 2^-53 x 1 rad = 2^-22."""
    import exact_attention_27_gb300 as fa
    g = torch.Generator().manual_seed(1)
    n = 256
    x = torch.randn(1, 2, n, 64, generator=g).to(torch.bfloat16)
    positions = (2 ** 31 - 1 - torch.randint(0, 10 ** 6, (1, 1, n), generator=g)).to(torch.int32)
    positions[0, 0, 1] = -2 ** 31
    inv = inv_freq(64)
    rotary = fa.Rotary(inv.cuda())
    y, _ = fa.rotary_forward(x.cuda(), None, positions.cuda(), rotary)
    # the 64-bit angle itself: the product is exact (24 + 31 bits and the sign: 55 > 53, so
    # reduced by hand modulo 2 pi in two parts)
    high, low = positions.long() // 65536 * 65536, positions.long() % 65536
    two_pi = 2 * math.pi
    axis = torch.zeros(32)
    a = torch.remainder(angles64(high, inv, axis), two_pi) + angles64(low, inv, axis)
    want, slack = turn64(x.double(), a[:, None], 64, False)
    # 2 pi itself in 64 bits is off by 2^-53 relative, 2^31 / 2 pi turns of it: 2^-22 as well
    err = (y.cpu().double() - want).abs()
    assert torch.all(err <= BF16 * want.abs() + 2 * slack)


@pytest.mark.parametrize("kind", ["fused", "in place", "broadcast", "token major out"])
def test_strides(kind):
    import exact_attention_27_gb300 as fa
    B, Hq, Hkv, N, d = 2, 4, 2, 33, 64
    g = torch.Generator().manual_seed(3)
    x = torch.randn(B, N, Hq + Hkv, d, generator=g).to(torch.bfloat16)
    q, k = x[:, :, :Hq].transpose(1, 2), x[:, :, Hq:].transpose(1, 2)
    xc = x.cuda()
    qc, kc = xc[:, :, :Hq].transpose(1, 2), xc[:, :, Hq:].transpose(1, 2)
    positions = torch.randint(0, 5000, (1, 1, N), generator=g).to(torch.int32).expand(1, B, N)
    pc = positions[:, :1].cuda().expand(1, B, N)
    inv = inv_freq(d)
    rotary = fa.Rotary(inv.cuda())
    if kind == "in place":
        qo, ko = qc, kc
        fa.fa_rotary(qc, qo, kc, ko, pc, rotary)
    elif kind == "broadcast":
        k = k[:, :1].expand(B, Hkv, N, d)
        qo, ko = fa.rotary_forward(qc, kc[:, :1].expand(B, Hkv, N, d), pc, rotary)
        assert 0 not in ko.stride()
    elif kind == "token major out":
        out = torch.zeros(B, N, Hq + Hkv + 1, d, dtype=torch.bfloat16, device="cuda")
        qo, ko = out[:, :, :Hq].transpose(1, 2), out[:, :, Hq:-1].transpose(1, 2)
        fa.fa_rotary(qc, qo, kc, ko, pc, rotary)
        assert torch.all(out[:, :, -1] == 0)
    else:
        qo, ko = fa.rotary_forward(qc, kc, pc, rotary)
    torch.cuda.synchronize()
    axis = torch.zeros(d // 2)
    check(qo, q, positions, inv, axis, d, False)
    check(ko, k, positions, inv, axis, d, False)


def test_training_step_gradients():
    """rotary_forward, fa_forward, fa_backward, rotary_backward against the 64-bit gradient of
    the whole (grouped heads, time / height / width), and that against differences."""
    import exact_attention_27_gb300 as fa
    B, Hq, Hkv, N, d = 1, 4, 2, 160, 64
    g = torch.Generator().manual_seed(4)
    q, k, v, do = (torch.randn(B, h, N, d, generator=g).to(torch.bfloat16)
                   for h in (Hq, Hkv, Hkv, Hq))
    t = torch.arange(N)
    positions = torch.stack((t // 16, t % 16 // 4, t % 4))[:, None].to(torch.int32)
    axis = torch.tensor([0] * 8 + [1] * 12 + [2] * 12)
    inv = inv_freq(d)
    rotary = fa.Rotary(inv.cuda(), (8, 12, 12))
    angle = angles64(positions, inv, axis)[:, None]
    scale = 1 / math.sqrt(d)

    def loss64(q, k, v):
        qr, kr = turn64(q, angle, d, False)[0], turn64(k, angle, d, False)[0]
        s = qr @ kr.repeat_interleave(Hq // Hkv, 1).transpose(2, 3) * scale
        s = s.masked_fill(torch.ones(N, N).triu(1).bool(), -math.inf)
        o = torch.softmax(s, -1) @ v.repeat_interleave(Hq // Hkv, 1)
        return (o * do.double()).sum()

    leaves = [x.double().requires_grad_() for x in (q, k, v)]
    want = torch.autograd.grad(loss64(*leaves), leaves)
    for x, grad in zip(leaves, want):
        step = torch.randn(x.shape, generator=g, dtype=torch.float64)
        with torch.no_grad():
            ahead = [y + 1e-5 * step if y is x else y for y in leaves]
            back = [y - 1e-5 * step if y is x else y for y in leaves]
            slope = (loss64(*ahead) - loss64(*back)) / 2e-5
        assert abs(slope - (grad * step).sum()) <= 1e-6 * grad.norm() * step.norm()

    qr, kr = fa.rotary_forward(q.cuda(), k.cuda(), positions.cuda(), rotary)
    vc = v.cuda()
    o, lse = fa.attention_forward(qr, kr, vc, causal=True)
    dqr, dkr, dv = fa.attention_backward(qr, kr, vc, o, lse, do.cuda(), causal=True)
    dq, dk = fa.rotary_backward(dqr, dkr, positions.cuda(), rotary)
    torch.cuda.synchronize()
    for got, ref in zip((dq, dk, dv), want):
        err = (got.cpu().double() - ref).abs().max()
        assert err <= 5e-2 * ref.abs().max(), err  # the backward's tolerance (parity.GRAD_REL)


def test_graph_replays_new_values():
    import exact_attention_27_gb300 as fa
    inv = inv_freq(64)
    rotary = fa.Rotary(inv.cuda())
    x = torch.randn(1, 4, 50, 64).to(torch.bfloat16)
    xc, pos = x.cuda(), torch.zeros(1, 1, 50, dtype=torch.int32, device="cuda")
    fa.rotary_forward(xc, None, pos, rotary)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        y, _ = fa.rotary_forward(xc, None, pos, rotary)
    pos.copy_(torch.arange(50, dtype=torch.int32)[None, None])
    graph.replay()
    torch.cuda.synchronize()
    check(y, x, torch.arange(50)[None, None], inv, torch.zeros(32), 64, False)
