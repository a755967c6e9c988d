"""Paged attention where few bits would show: weights far below the largest, and long histories
at the largest head dimension."""

import math

import pytest
import torch

from paged_plain import BF16, F16, F32, Step, attention64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def bounds(o, lse, a, size, d, lost, e4m3):
    """Largest |error| of o [n, H, d] and lse [n, H], 64-bit values with attention64's a and size.
    Scores and exponentials as in attention_bounds: delta, once in every p and once in the sum.
    P: half a step of its format (bf16 2^-8, fp16 2^-11 of each p); `lost` [n, H, d]: what the
    absolute half step of fp16 below 2^-14 can come to.  O: half a step."""
    delta = (d + 8) * F32 * (size + lse.abs()) + 2.0 ** -20
    p = F16 if e4m3 else BF16
    o_tol = BF16 * o.abs() * (1 + 2.0 ** -6) + (p + 2 * delta[..., None]) * a
    if e4m3:
        o_tol = o_tol + lost * (1 + 2.0 ** -6)
    return o_tol + 1e-30, 2 * delta + 2 * F32 * lse.abs()


def compare(o, lse, want, d, lost, e4m3):
    ro, rl, a, size = want
    ot, lt = bounds(ro, rl, a, size, d, lost, e4m3)
    err, lerr = (o.cpu().double() - ro).abs(), (lse.cpu().double() - rl).abs()
    assert torch.all(err <= ot), f"o off by {(err / ot).max().item():.2f} of the bound"
    assert torch.all(lerr <= lt), f"lse off by {(lerr / lt).max().item():.2f} of the bound"


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("n", [1, 20, 40])
@pytest.mark.parametrize("gap", [10, 14, 17, 19])
def test_weights_far_below_the_largest(gap, n, d, e4m3):
    """Every 16th key is `gap` nats above the others and has a value of zero, so that o is what
    the others' small weights make of it.  The largest p of every group of keys with a running
    maximum of its own is 2^7 for 8-bit pages (the keys above share one score, and each group
    begins with one), and half of fp16's smallest step is 2^-25: each weight is off by 2^-25 / L,
    L = 2^7 exp(lse - that score), at most."""
    import exact_attention_27_gb300 as fa
    m, G, page = 3001, 4, 64
    g = torch.Generator().manual_seed(gap + d + n)
    k = torch.randn(m, 1, d, generator=g)
    k[:, :, 0] = 16.0 - gap
    k[::16] = 0.0
    k[::16, :, 0] = 16.0
    v = 1.0 + 0.25 * torch.randn(m, 1, d, generator=g)
    v[::16] = 0.0
    q = 0.1 * torch.randn(n, G, d, generator=g)
    q[..., 0] = math.sqrt(d)
    q = q.to(torch.bfloat16)
    kd, vd = (0.0625, 0.125) if e4m3 else (1.0, 1.0)
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    n_pages = -(-m // page)
    pages, stored = [], []
    for x, ds in ((k, kd), (v, vd)):
        x = (x / ds).to(dtype)
        stored.append(x.double() * ds)
        room = torch.full((n_pages * page, 1, d), float("nan"))
        room[:m] = x.float()
        pages.append(room.view(n_pages, page, 1, d).transpose(1, 2).contiguous().to(dtype).cuda())
    cache = fa.PagedCache(pages[0], pages[1], kd, vd)
    batch = fa.PagedBatch(torch.arange(n_pages, dtype=torch.int32, device="cuda")[None],
                          torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                          torch.tensor([m], dtype=torch.int32, device="cuda"), n)
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.paged_attention(cache, batch, q.cuda(), True, scale)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    k64, v64 = stored
    q64 = q.double()
    want = attention64(q64, k64, v64, scale, True, m - n)
    top = scale * (q64 @ k64[0, 0])
    lost = 2.0 ** -25 * v64.abs().sum(0)[None] / (2.0 ** 7 * torch.exp(want[1] - top))[..., None]
    compare(o, lse, want, d, lost, e4m3)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 20, 100])
@pytest.mark.parametrize("d", [128, 256])
def test_long_histories(d, n, e4m3):
    """Tens of thousands of keys of one head.  The largest p of a group of keys with a running
    maximum of its own is 2^7 at least for 8-bit pages: each of m weights is off by 2^-32 of the
    sum at most where fp16 ends."""
    import exact_attention_27_gb300 as fa
    m = 33001 + 7 * n
    step = Step([n], [m], 2, 1, d, 64, e4m3, seed=d + n)
    cache, batch = step.handles()
    scale = 1.0 / math.sqrt(d)
    o, lse = fa.paged_attention(cache, batch, step.q, True, scale)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    want = attention64(step.q_cpu.double(), step.k64[0], step.v64[0], scale, True, m - n)
    compare(o, lse, want, d, m * 2.0 ** -32 * step.v64[0].abs().max(), e4m3)


@pytest.mark.parametrize("q_lens,kv_lens", [([1, 1], [3000, 200]), ([20, 300], [3000, 400])])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("power", [-126, -60, 110])
def test_descales_at_the_ends_of_fp32(power, d, q_lens, kv_lens):
    """A factor of V near the smallest and largest of its range, with many keys of like weight:
    the factor over the weights' sum lies outside fp32 where the output does not.  o is that of a
    factor of 1 times the factor, exactly: a power of two."""
    import exact_attention_27_gb300 as fa
    step = Step(q_lens, kv_lens, 4, 2, d, 16, True, seed=d, k_scale=0.01)
    batch = step.handles()[1]
    outs = []
    for descale in (1.0, 2.0 ** power):
        cache = fa.PagedCache(step.k_pages, step.v_pages, step.kd, descale)
        outs.append(fa.paged_attention(cache, batch, step.q))
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    (a, la), (b, lb) = outs
    assert torch.equal(la, lb)
    want = a.double() * 2.0 ** power
    # Below 2^-126 bf16 has steps of 2^-133, half of which is 2^-134; a itself is off by 2^-9 of
    # what is then below 2^-126, and fp32's steps there are 2^-149: 2^-134 + 2^-135 + 2^-150.
    # From 2^-126 on both are the same bits, scaled.
    slack = torch.where(want.abs() < 2.0 ** -126, 2.0 ** -133, 0.0)
    assert torch.all((b.double() - want).abs() <= slack)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("n", [1, 20, 130])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("base", [0, 20, 22, 23, 24, 25, 26, 27])
def test_far_scores_that_climb(base, d, n, e4m3):
    """Scores of 2^base that climb by a few nats a tile, where fp32's steps at that size (2^base
    x 2^-23) are no longer small beside them.  With values of 1 o is 1, however the weights come
    out: their sum, rounded (2^-11 or 2^-8 of each weight), over their sum, and half a step of
    o.  lse is off by what the scores are: a few steps of their size."""
    import exact_attention_27_gb300 as fa
    S, H, m, page = 64, 8, 1500, 64
    g = torch.Generator().manual_seed(base + d + n)
    k = torch.zeros(m, H, d)
    k[:, :, 0] = 16.0 if base else 0.0
    climb = torch.linspace(-15.0, 15.0, m)[:, None] + 4.0 * torch.rand(m, H, generator=g)
    k[:, :, 1] = climb.clamp(-16.0, 16.0)
    kd = 0.0625 if e4m3 else 1.0
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    k = (k / kd).to(dtype)
    n_pages = -(-m // page)
    pages = []
    for x in (k.float(), torch.ones(m, H, d)):
        room = torch.full((n_pages * page, H, d), float("nan"))
        room[:m] = x
        pages.append(room.view(n_pages, page, H, d).transpose(1, 2).contiguous().to(dtype).cuda())
    cache = fa.PagedCache(pages[0], pages[1], kd, 1.0)
    # (every sequence reads the same pages)
    table = torch.arange(n_pages, dtype=torch.int32, device="cuda").expand(S, n_pages)
    starts = torch.arange(0, n * S + 1, n, dtype=torch.int32, device="cuda")
    batch = fa.PagedBatch(table, starts, torch.full((S,), m, dtype=torch.int32, device="cuda"), n)
    q = torch.zeros(n * S, H, d)
    q[..., 0] = 2.0 ** (base - 4)
    q[..., 1] = 3.0
    o, lse = fa.paged_attention(cache, batch, q.to(torch.bfloat16).cuda(), False, 1.0)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    assert torch.isfinite(o).all() and torch.isfinite(lse).all()
    # (the weights' rounding 2^-8 or 2^-11, sums of at most m terms in fp32, o's rounding)
    tol = (F16 if e4m3 else BF16) + BF16 + 2 * m * F32
    assert (o.float() - 1.0).abs().max().item() <= tol
    top = 2.0 ** (base - 4) * 16.0 * bool(base)
    want = top + torch.logsumexp(3.0 * kd * k[:, :, 1].double(), 0)
    size = top + 3.0 * 16.0
    err = (lse.cpu().double().view(S, n, H) - want).abs().max().item()
    assert err <= 2 * ((d + 8) * F32 * 2 * size + 2.0 ** -20) + 2 * F32 * size
