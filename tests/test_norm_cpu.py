"""Norms of heads' rows on the host: refusals, and the 64-bit values against differences."""

import ctypes

import pytest
import torch

import exact_attention_27_gb300 as fa
from exact_attention_27_gb300 import _build, _lib
from norm_plain import backward64, forward64
from test_paged_cpu import F, P, Q, batch, cache, rows, spec


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.library()


def norm(q=P, k=P, dtype=0, eps=1e-6):
    return _lib.HeadNormStruct(q, k, dtype, eps)


def forward(lib, q=None, k=None, B=2, N=8, d=64, pos=P, axis=16, stride=8, s=None, n=None):
    ref = ctypes.byref
    return lib.fa_norm_rotary(ref(q) if q is not None else ref(rows()), ref(k) if k else None, B, N,
                              d, ref(n or norm()), pos, axis, stride,
                              None if s is False else ref(s or spec()), None)


def backward(lib, dq=None, dk=None, q=None, k=None, d=64, n=None, dqw=P, dkw=None, ws=P,
             bytes=2 ** 40, s=None, pos=P):
    ref = ctypes.byref
    return lib.fa_norm_rotary_backward(
        ref(dq or rows()), ref(dk) if dk else None, ref(q or rows()), ref(k) if k else None, 2, 8,
        d, ref(n or norm()), dqw, dkw, pos, 16, 8, ref(s or spec()), ws, bytes, None)


BAD_NORMS = [norm(q=Q), norm(k=Q), norm(dtype=2), norm(dtype=-1), norm(eps=0.0), norm(eps=-1.0),
             norm(eps=float("nan")), norm(eps=float("inf"))]


@pytest.mark.parametrize("n", BAD_NORMS)
def test_bad_norms_are_rejected(lib, n):
    ref = ctypes.byref
    assert forward(lib, n=n) == fa.FA_ERR_INVALID_ARGUMENT
    assert backward(lib, n=n) == fa.FA_ERR_INVALID_ARGUMENT
    assert lib.fa_paged_append_norm(ref(cache()), ref(batch()), P, 128, 64, P, 128, 64, 2, P, 256,
                                    64, P, 256, 64, 4, ref(n), None, None, 0,
                                    None) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(B=0), dict(N=0), dict(pos=None), dict(pos=F), dict(axis=-1), dict(stride=-8),
    dict(q=rows(in_=None)), dict(q=rows(out=Q)), dict(q=rows(heads=0)), dict(q=rows(in_pos=60)),
    dict(q=rows(out_pos=0)), dict(k=rows(heads=0)), dict(B=2 ** 20, N=2 ** 20),
    dict(s=spec(rot_dim=80)), dict(s=spec(axes=0))])
def test_forward_rejects(lib, kw):
    assert forward(lib, **kw) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(q=rows(in_=None)), dict(q=rows(in_=Q)), dict(q=rows(heads=3)), dict(q=rows(in_head=4)),
    dict(q=rows(in_pos=-8)), dict(dk=rows()), dict(k=rows()), dict(dkw=P), dict(dqw=F),
    dict(dk=rows(), k=rows(), dkw=F), dict(ws=None), dict(ws=Q), dict(bytes=0), dict(pos=None),
    dict(dq=rows(out=None))])
def test_backward_rejects(lib, kw):
    assert backward(lib, **kw) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("d", [0, 32, 80, 512])
def test_unsupported_head_dim(lib, d):
    assert forward(lib, d=d) == fa.FA_ERR_UNSUPPORTED
    assert forward(lib, d=d, s=False, pos=None) == fa.FA_ERR_UNSUPPORTED
    assert backward(lib, d=d) == fa.FA_ERR_UNSUPPORTED
    assert lib.fa_norm_rotary_backward_workspace_bytes(d) == 0


def test_append_with_nothing_to_do_needs_no_gpu(lib):
    ref = ctypes.byref
    assert lib.fa_paged_append_norm(ref(cache(k=None, v=None)), ref(batch(S=0)), None, 128, 64,
                                    None, 128, 64, 2, None, 0, 0, None, 0, 0, 0, ref(norm()), None,
                                    None, 0, None) == fa.FA_OK


def test_handles_check_their_tensors():
    for kw in (dict(q_weight=torch.zeros(64)), dict(k_weight=torch.zeros(64)), dict(eps=0.0),
               dict(eps=float("nan"))):
        with pytest.raises(ValueError):
            fa.HeadNorm(**kw)


@pytest.mark.parametrize("interleaved", [False, True])
def test_values_against_differences(interleaved):
    g = torch.Generator().manual_seed(2)
    x, dy = (torch.randn(3, 2, 16, generator=g, dtype=torch.float64) for _ in range(2))
    w = torch.randn(16, generator=g, dtype=torch.float64)
    angle = torch.randn(3, 1, 4, generator=g, dtype=torch.float64)
    eps = 0.1
    dx, dw, _, _ = backward64(x, w, eps, dy, angle, 8, interleaved)

    def value():
        return (forward64(x, w, eps, angle, 8, interleaved)[0] * dy).sum()
    h = 1e-6
    for t, grad, places in ((x, dx, [(0, 0, 0), (1, 1, 5), (2, 0, 9), (2, 1, 15)]),
                            (w, dw, [(0,), (3,), (7,), (12,)])):
        for at in places:
            keep = t[at].item()
            f = []
            for e in (h, -h):
                t[at] = keep + e
                f.append(value())
            t[at] = keep
            assert abs((f[0] - f[1]) / (2 * h) - grad[at]) < 1e-7 * (1 + abs(grad[at]))


@pytest.mark.parametrize("mistake", ["mean over rot", "eps outside", "weight after turn",
                                     "turn sign", "no mean term", "weight missing in mean"])
def test_bounds_notice_mistakes(mistake):
    g = torch.Generator().manual_seed(3)
    d, rot, eps = 64, 32, 0.3
    x, dy = (torch.randn(20, 2, d, generator=g).to(torch.bfloat16).double() for _ in range(2))
    w = 1 + 0.3 * torch.randn(d, generator=g, dtype=torch.float64)
    angle = torch.randn(20, 1, rot // 2, generator=g, dtype=torch.float64)
    y, slack = forward64(x, w, eps, angle, rot)
    tol = 2.0 ** -8 * (y.abs() + slack) + slack
    dx, dw, dx_tol, dw_tol = backward64(x, w, eps, dy, angle, rot)
    worst = 0.0
    if mistake == "mean over rot":
        r = (x[..., :rot].square().mean(-1, keepdim=True) + eps).rsqrt()
        bad = forward64(x, w, 0.0, angle, rot)[0] * (x.square().mean(-1, keepdim=True)).sqrt() * r
        worst = ((bad - y).abs() / tol).max()
    elif mistake == "eps outside":
        bad = y * (x.square().mean(-1, keepdim=True) + eps).sqrt() / (
            x.square().mean(-1, keepdim=True).sqrt() + eps)
        worst = ((bad - y).abs() / tol).max()
    elif mistake == "weight after turn":
        bad = forward64(x, torch.ones_like(w), eps, angle, rot)[0] * w
        worst = ((bad - y).abs() / tol).max()
    elif mistake == "turn sign":
        bad = backward64(x, w, eps, dy, -angle, rot)
        worst = min(((bad[0] - dx).abs() / dx_tol).max(), ((bad[1] - dw).abs() / dw_tol).max())
    else:
        one = torch.ones_like(w)
        r = (x.square().mean(-1, keepdim=True) + eps).rsqrt()
        u = x * r
        turned = backward64(x, one, eps, dy, angle, rot)
        gu = turned[0] / r  # g - u mean(g o u)
        if mistake == "no mean term":
            bad = r * (gu * w)
        else:
            bad = turned[0] * w
        worst = ((bad - dx).abs() / dx_tol).max()
        assert u.shape == dx.shape
    assert worst > 3, worst
