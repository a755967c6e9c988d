"""A server's steps, append and then attention, against 64-bit values over the very bits that
each call reads."""

import pytest
import torch

import paged_steps as ps

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_steps_over_what_is_stored(e4m3):
    """After each append the returned q and the new rows of the pages are one rounding from the
    turned inputs, every older row keeps its bits, and the attention is that of the returned q
    over the stored rows: no rounding is left to allow for but its own."""
    import exact_attention_27_gb300 as fa
    S, n_pages = len(ps.TOTAL), 40
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kd, vd = (0.125, 0.0625) if e4m3 else (1.0, 1.0)
    pages = [torch.full((n_pages, ps.HKV, ps.PAGE, ps.D), float("nan"), device="cuda").to(dtype)
             for _ in range(2)]
    cache = fa.PagedCache(pages[0], pages[1], kd, vd)
    order = torch.randperm(n_pages, generator=torch.Generator().manual_seed(6))[:10 * S].view(S, 10)
    table = order.to(torch.int32).cuda()
    rotary = fa.Rotary(ps.INV_FREQ.cuda())
    data = ps.inputs()

    def rows(x, s, m):
        """The first m rows of sequence s, [m, HKV, D]."""
        return x.cpu().float()[order[s]].transpose(1, 2).reshape(-1, ps.HKV, ps.D)[:m]

    done, held = [0] * S, {}
    for new in ps.STEPS:
        before, done = done, [a + n for a, n in zip(done, new)]
        q, k, v = (torch.cat([data[s][i][before[s]:done[s]] for s in range(S)]).cuda()
                   for i in range(3))
        starts = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32).cuda()
        batch = fa.PagedBatch(table, starts, torch.tensor(done, dtype=torch.int32).cuda(),
                              max(new))
        q = fa.paged_append(cache, batch, k, v, rotary, q=q)
        o, lse = fa.paged_attention(cache, batch, q)
        torch.cuda.synchronize()
        assert fa.fa_last_device_error() == 0
        q, o, lse = q.cpu().double(), o.cpu().double(), lse.cpu().double()
        at = 0
        for s, n in enumerate(new):
            a, m = before[s], done[s]
            stored = [rows(x, s, m) for x in pages]
            for i, x in enumerate(stored):
                assert a == 0 or torch.equal(x[:a], held[s, i][:a])
                held[s, i] = x
            if n == 0:
                continue
            want, slack = ps.turned(data[s][0][a:m], a)
            assert torch.all((q[at:at + n] - want).abs() <=
                             ps.stored_bound(want, slack, 1.0, False))
            want, slack = ps.turned(data[s][1][a:m], a)
            assert torch.all((stored[0][a:].double() - want / kd).abs() <=
                             ps.stored_bound(want, slack, kd, e4m3))
            want = data[s][2][a:m].double()
            assert torch.all((stored[1][a:].double() - want / vd).abs() <=
                             ps.stored_bound(want, torch.zeros_like(want), vd, e4m3))
            v64 = stored[1].double() * vd
            ro, rl, ra, size = ps.exact(q[at:at + n], stored[0].double() * kd, v64)
            ot, lt = ps.attention_bound(ro, rl, ra, size, m, v64.abs().max(), e4m3)
            err, lerr = (o[at:at + n] - ro).abs(), (lse[at:at + n] - rl).abs()
            assert torch.all(err <= ot), f"o off by {(err / ot).max().item():.2f} of the bound"
            assert torch.all(lerr <= lt), f"lse off by {(lerr / lt).max().item():.2f} of the bound"
            at += n
