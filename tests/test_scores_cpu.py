"""Shaped scores on the host: refusals, and what the tests of the kernels rest on."""

import ctypes
import math

import pytest
import torch

import exact_attention_27_gb300 as fa
from exact_attention_27_gb300 import _build, _lib
from scores_plain import Head, off_by, spans_of, whole

# Fake, 16-byte aligned, never dereferenced: validation fails before any use.
P = 0x10000
Q = 0x10008  # 8-byte aligned only
F = 0x10002  # 2-byte aligned only


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.library()


def spec(softcap=0.0, slopes=None, window=0):
    return _lib.ScoreSpec(softcap, slopes, window)


def spans(first=P, end=P, stride=64):
    return _lib.KeySpansStruct(first, end, stride)


def call(lib, backward=False, s=None, r=None, **kw):
    a = dict(q=P, k=P, v=P, o=P, lse=P, do=P, dq=P, dk=P, dv=P, B=1, Hq=2, Hkv=1, Nq=64, Nkv=64,
             d=64, scale=0.125, causal=1, off=0, ws=P, bytes=2 ** 40)
    a.update(kw)
    p = ctypes.c_void_p
    head = [p(a[x]) if a[x] else None for x in ("q", "k", "v", "o", "lse")]
    if backward:
        head += [p(a[x]) if a[x] else None for x in ("do", "dq", "dk", "dv")]
    fn = lib.fa_backward_scores if backward else lib.fa_forward_scores
    work = [p(a["ws"]) if a["ws"] else None, a["bytes"]] if backward else []
    return fn(*head, a["B"], a["Hq"], a["Hkv"], a["Nq"], a["Nkv"], a["d"],
              ctypes.c_float(a["scale"]), a["causal"], a["off"],
              ctypes.byref(s) if s is not None else None,
              ctypes.byref(r) if r is not None else None, *work, None)


BAD = [dict(q=None), dict(k=None), dict(v=None), dict(o=None), dict(lse=None), dict(q=Q), dict(o=Q),
       dict(lse=F), dict(B=0), dict(Hq=3, Hkv=2), dict(Nq=0), dict(Nkv=0), dict(Nkv=-4),
       dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")), dict(scale=3e38),
       dict(causal=2), dict(off=-1), dict(off=2 ** 31 - 20), dict(Nkv=2 ** 31 - 100),
       dict(s=spec(-1.0)), dict(s=spec(float("nan"))), dict(s=spec(float("inf"))),
       dict(s=spec(1e-40)), dict(s=spec(3e38)), dict(s=spec(1e-30), scale=1e20),
       dict(s=spec(1e30), scale=1e-20), dict(s=spec(slopes=F)), dict(s=spec(window=-1)),
       dict(r=spans(first=F)), dict(r=spans(end=F)), dict(r=spans(stride=-64))]


@pytest.mark.parametrize("kw", BAD)
@pytest.mark.parametrize("backward", [False, True])
def test_bad_calls_are_rejected(lib, kw, backward):
    assert call(lib, backward, **kw) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [dict(do=None), dict(dq=None), dict(dk=None), dict(dv=Q),
                                dict(do=Q), dict(ws=None), dict(ws=Q), dict(bytes=64)])
def test_backward_rejects(lib, kw):
    assert call(lib, True, **kw) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("d", [0, 32, 80, 192, 512])
@pytest.mark.parametrize("backward", [False, True])
def test_unsupported_head_dim(lib, d, backward):
    assert call(lib, backward, d=d) == fa.FA_ERR_UNSUPPORTED


@pytest.mark.parametrize("args", [(0, 2, 1, 64, 64, 64, 1, 0), (1, 3, 2, 64, 64, 64, 1, 0),
                                  (1, 2, 1, 0, 64, 64, 1, 0), (1, 2, 1, 64, 0, 64, 1, 0),
                                  (1, 2, 1, 64, 64, 80, 1, 0), (1, 2, 1, 64, 64, 64, 2, 0),
                                  (1, 2, 1, 64, 64, 64, 1, -1)])
def test_workspace_rejects(lib, args):
    assert lib.fa_backward_scores_workspace_bytes(*args) == 0


def test_handles_check_their_arguments():
    for kw in (dict(softcap=-1.0), dict(softcap=float("nan")), dict(softcap=float("inf")),
               dict(window=-1), dict(window=2 ** 31), dict(slopes=torch.zeros(4)),
               dict(slopes=torch.zeros(4, dtype=torch.bfloat16))):
        with pytest.raises(ValueError):
            fa.Scores(**kw)
    with pytest.raises(ValueError):
        fa.KeySpans()
    for bad in (torch.zeros(2, 8, dtype=torch.int32), torch.zeros(2, 8, dtype=torch.int64), [1, 2]):
        with pytest.raises(ValueError):
            fa.KeySpans(bad)
    x = torch.zeros(1, 2, 8, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.fa_forward_scores(x, x, x, x, torch.zeros(1, 2, 8), 0.1, True)


# ------------------------------------------------------------------ what the GPU tests rest on

def inputs(n=9, m=12, d=8, seed=0):
    g = torch.Generator().manual_seed(seed)
    return [torch.randn(s, d, generator=g, dtype=torch.float64) for s in (n, m, m, n)]


KINDS = [dict(), dict(softcap=2.0), dict(slope=0.3), dict(softcap=1.5, slope=0.1, q_offset=3)]


@pytest.mark.parametrize("kw", KINDS)
@pytest.mark.parametrize("causal", [False, True])
def test_gradients_against_differences(kw, causal):
    q, k, v, do = inputs()
    off = kw.get("q_offset", 3)
    see = spans_of(9, 12, causal, off, end=torch.tensor([12] * 7 + [0, 4]))
    x = Head(q, k, v, see, 0.4, do=do, **kw)
    assert not x.live[7] and torch.all(x.o[7] == 0) and torch.all(x.dq[7] == 0)
    eps = 1e-6
    for t, grad in ((q, x.dq), (k, x.dk), (v, x.dv)):
        for at in ((0, 0), (2, 5), (6, 3), (8, 7)):
            keep = t[at].item()
            f = []
            for e in (eps, -eps):
                t[at] = keep + e
                f.append((Head(q, k, v, see, 0.4, **kw).o * do).sum())
            t[at] = keep
            diff = (f[0] - f[1]) / (2 * eps)
            # the differences' own error: eps^2 times a third derivative, and rounding over eps
            assert abs(diff - grad[at]) < 1e-7 * (1 + abs(diff))


@pytest.mark.parametrize("mistake", ["no cap gradient", "cap after slopes", "slope sign",
                                     "distance off by one", "window off by one", "span end",
                                     "no scale on dk", "lse before the cap", "group sum"])
def test_bounds_notice_mistakes(mistake):
    """The bounds of the GPU tests are far below what a slip in the formulas does."""
    g = torch.Generator().manual_seed(1)
    B, Hq, Hkv, n, d = 1, 4, 2, 150, 64
    q, k, v, do = (torch.randn(B, h, n, d, generator=g).to(torch.bfloat16)
                   for h in (Hq, Hkv, Hkv, Hq))
    q = q * 3
    slopes = torch.tensor([0.25, 0.06, 0.016, 0.004])
    cap, window, scale = 8.0, 40, 1 / 8
    end = torch.full((n,), n - 20)
    see = [spans_of(n, n, True, 0, window, end=end)]
    val, tol = whole(q, k, v, see, scale, cap, slopes, do=do)
    kw = dict(see=see, scale=scale, softcap=cap, slopes=slopes, do=do)
    if mistake == "slope sign":
        kw["slopes"] = -slopes
    elif mistake == "distance off by one":  # shifts all scores of a row alike but at the diagonal
        kw["q_offset"] = 1
        kw["see"] = see
    elif mistake == "window off by one":
        kw["see"] = [spans_of(n, n, True, 0, window + 1, end=end)]
    elif mistake == "span end":
        kw["see"] = [spans_of(n, n, True, 0, window, end=end + 1)]
    elif mistake == "lse before the cap":
        kw["softcap"] = 0.0
    got, _ = whole(q, k, v, **kw)
    if mistake == "no cap gradient":
        plain = Head(q[0, 0].double(), k[0, 0].double(), v[0, 0].double(), see[0], scale, cap,
                     0.25, do=do[0, 0].double())
        assert off_by(plain.dq, plain.dq, plain.dq_tol) <= 1
        x = q[0, 0].double() @ k[0, 0].double().T * scale
        p = torch.exp((cap * torch.tanh(x / cap) - 0.25 * (torch.arange(n)[:, None] - torch.arange(
            n)).abs()).masked_fill(~see[0], -math.inf) - plain.lse.masked_fill(
                ~plain.live, 0.0)[:, None])
        dp = do[0, 0].double() @ v[0, 0].double().T
        dq = p * (dp - (p * dp).sum(1, keepdim=True)) @ k[0, 0].double() * scale
        assert off_by(dq, plain.dq, plain.dq_tol) > 3
        return
    if mistake == "cap after slopes":
        x = Head(q[0, 0].double(), k[0, 0].double(), v[0, 0].double(), see[0], scale, cap, 0.25)
        raw = q[0, 0].double() @ k[0, 0].double().T * scale - 0.25 * (
            torch.arange(n)[:, None] - torch.arange(n)).abs()
        s = (cap * torch.tanh(raw / cap)).masked_fill(~see[0], -math.inf)
        assert off_by(torch.logsumexp(s, 1), x.lse, x.lse_tol) > 3
        return
    if mistake == "no scale on dk":
        got["dk"] = got["dk"] / scale
    if mistake == "group sum":
        one, _ = whole(q[:, ::2], k, v, see, scale, cap, slopes[::2], do=do[:, ::2])
        got["dk"], got["dv"] = one["dk"], one["dv"]
    worst = max(off_by(got[a], val[a], tol[a]) for a in val)
    if mistake == "distance off by one":
        # (a causal row's scores all fall by the slope: lse alone shows it)
        assert off_by(got["lse"], val["lse"], tol["lse"]) > 3
    assert worst > 3, worst


# ------------------------------------------------------------------ over a paged cache

def paged(lib, s, c=None, **kw):
    from test_paged_cpu import batch, cache
    a = dict(q=P, qt=256, qh=64, o=P, ot=256, oh=64, lse=P, T=2, Hq=4, scale=0.125, causal=1, ws=P,
             bytes=2 ** 40)
    a.update(kw)
    ref = ctypes.byref
    return lib.fa_forward_paged_scores(
        ref(c or cache()), ref(batch()), a["q"], a["qt"], a["qh"], a["o"], a["ot"], a["oh"],
        a["lse"], a["T"], a["Hq"], ctypes.c_float(a["scale"]), a["causal"],
        None if s is None else ref(s), a["ws"], a["bytes"], None)


@pytest.mark.parametrize("s", [spec(-1.0), spec(float("nan")), spec(float("inf")), spec(1e-40),
                               spec(3e38), spec(slopes=F), spec(window=-1)])
def test_paged_rejects_bad_scores(lib, s):
    assert paged(lib, s) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [dict(q=None), dict(o=Q), dict(lse=F), dict(T=-1), dict(Hq=3),
                                dict(scale=0.0), dict(causal=2), dict(qt=4), dict(ot=0)])
def test_paged_rejects(lib, kw):
    assert paged(lib, spec(10.0), **kw) == fa.FA_ERR_INVALID_ARGUMENT


def test_paged_with_nothing_to_do_needs_no_gpu(lib):
    assert paged(lib, spec(10.0), T=0, q=None, o=None, ws=None) == fa.FA_OK
    assert paged(lib, None, T=0, q=None, o=None, ws=None) == fa.FA_OK
