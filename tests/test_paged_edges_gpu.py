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


def padded(x, pad, fill=float("nan")):
    """x as a view whose rows lie `pad` values further apart, with `fill` between them."""
    wide = torch.full((*x.shape[:-1], x.shape[-1] + pad), fill, device=x.device).to(x.dtype)
    raw = torch.uint8 if x.element_size() == 1 else torch.int16
    wide.view(raw)[..., :x.shape[-1]] = x.view(raw)
    return wide[..., :x.shape[-1]]


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("q_lens", [[1, 2, 1], [1, 70, 300]])
def test_rows_apart(q_lens, d, e4m3):
    """Rows of pages, q and o 16 bytes further apart than dense ones (so that some start on no
    32-byte boundary), with NaN between them; a block table that is a slice of a wider one."""
    import exact_attention_27_gb300 as fa
    step = Step(q_lens, [90, 400, 3000], 4, 2, d, 16, e4m3, seed=d)
    pad = 16 if e4m3 else 8
    step.k_pages, step.v_pages = padded(step.k_pages, pad), padded(step.v_pages, pad)
    wide = torch.full((3, step.table.shape[1] + 9), -1, dtype=torch.int32, device="cuda")
    wide[:, 4:-5] = step.table
    step.table = wide[:, 4:-5]
    cache, batch = step.handles()
    q, o = padded(step.q, 8), padded(torch.zeros_like(step.q), 8, 3.0)
    lse = torch.empty(step.T, 4, device="cuda")
    scale = 1 / math.sqrt(d)
    ws = fa.paged_workspace(cache, batch, q)
    fa.fa_forward_paged(cache, batch, q, o, lse, scale, True, ws)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    step.check(o, lse, scale, True)
    around = o.as_strided((step.T, 4, 8), o.stride(), o.storage_offset() + d)
    assert torch.all(around == 3.0)
    fa.fa_forward_paged(cache, batch, q, o.zero_(), None, scale, True, ws)
    torch.cuda.synchronize()
    step.check(o, lse, scale, True)


@pytest.mark.parametrize("q_lens", [[1, 3], [50, 3]])
def test_rows_before_the_first_start(q_lens):
    """Starts that begin past row 0: the rows before belong to no sequence."""
    import exact_attention_27_gb300 as fa
    step = Step(q_lens, [80, 33], 4, 2, 64, 16, seed=4)
    lead = 5
    q = torch.cat([torch.randn(lead, 4, 64, device="cuda").to(torch.bfloat16), step.q])
    step.q_start += lead
    cache, batch = step.handles()
    o = torch.full_like(q, 7.0)
    lse = torch.full(q.shape[:2], 7.0, device="cuda")
    ws = fa.paged_workspace(cache, batch, q)
    fa.fa_forward_paged(cache, batch, q, o, lse, 0.1, True, ws)
    before = [x.clone() for x in (step.k_pages, step.v_pages)]
    k, v = (torch.cat([torch.ones(lead, 2, 64).to(torch.bfloat16)] +
                      [x[m - n:m].to(torch.bfloat16)
                       for x, n, m in zip(xs, step.q_lens, step.kv_lens)]).cuda()
            for xs in (step.k64, step.v64))
    q_out = torch.full_like(q, 7.0)
    fa.fa_paged_append(cache, batch, k, v, q=q, q_out=q_out)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    step.check(o[lead:], lse[lead:], 0.1, True)
    assert torch.all(o[:lead] == 7.0) and torch.all(lse[:lead] == 7.0)
    assert torch.all(q_out[:lead] == 7.0) and torch.equal(q_out[lead:], q[lead:])
    for now, was in zip((step.k_pages, step.v_pages), before):
        assert torch.equal(now.view(torch.int16), was.view(torch.int16))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("new", [[1, 1, 1], [1, 40, 0]])
def test_captured_serving_step(new, e4m3):
    """Append and attention in one graph on a stream of its own, replayed token after token with
    the lengths moved on in place, leave what the same calls leave one by one."""
    import exact_attention_27_gb300 as fa
    d, Hq, Hkv = 128, 8, 2
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    steps, T = 4, sum(new)
    g = torch.Generator().manual_seed(sum(new))
    xs = torch.randn(steps, T, Hq + 2 * Hkv, d, generator=g).to(torch.bfloat16).cuda()
    table = torch.randperm(60, generator=g)[:54].view(3, 18).to(torch.int32).cuda()
    starts = torch.tensor([0, new[0], new[0] + new[1], T], dtype=torch.int32).cuda()
    rotary = fa.Rotary((10000.0 ** (-torch.arange(64) / 64)).float().cuda())
    grow = torch.tensor(new, dtype=torch.int32).cuda()
    first = torch.randn(60, Hkv, 16, d, generator=g)

    def server():
        pages = [(first * f).to(dtype).cuda() for f in (4.0, 8.0)]
        lens = torch.tensor([100, 31, 5], dtype=torch.int32).cuda() + grow
        cache = fa.PagedCache(pages[0], pages[1], *((0.25, 0.125) if e4m3 else (1.0, 1.0)))
        batch = fa.PagedBatch(table, starts, lens, max(new))
        x = xs[0].clone()

        def step(stream=None):
            q = fa.paged_append(cache, batch, x[:, Hq:Hq + Hkv], x[:, Hq + Hkv:], rotary,
                                q=x[:, :Hq], stream=stream)
            return fa.paged_attention(cache, batch, q, stream=stream)
        return pages, lens, x, step

    pages, lens, x, step = server()
    want = []
    for i in range(steps):
        x.copy_(xs[i])
        want.append([t.clone() for t in step()])
        lens += grow
    want += [[p.view(torch.uint8).clone() for p in pages]]

    pages, lens, x, step = server()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    step(side)  # (stores the first step's rows, as the first replay does again)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    got = []
    for i in range(steps):
        x.copy_(xs[i])
        graph.replay()
        got.append([t.clone() for t in out])
        lens += grow
    got += [[p.view(torch.uint8).clone() for p in pages]]
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    for a, b in zip(want, got):
        for u, w in zip(a, b):
            assert torch.equal(u, w)


def test_positions_and_frequencies_in_wider_buffers():
    """Positions as slices of wider buffers, a row of them for every batch entry, frequencies
    behind others, on a stream of its own."""
    import exact_attention_27_gb300 as fa
    B, H, N, d, axes = 3, 4, 37, 128, 2
    x = torch.randn(B, H, N, d, device="cuda").to(torch.bfloat16)
    buffer = torch.randint(-500, 500, (4, B + 1, N + 11), dtype=torch.int32, device="cuda")
    freq = torch.rand(3 + d // 2, device="cuda")
    rotary = fa.Rotary(freq[3:], (20, 44))
    dense = fa.Rotary(freq[3:].clone(), (20, 44))
    view = buffer[1:3, 1:, 7:7 + N]
    want, _ = fa.rotary_forward(x, None, view.contiguous(), dense)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    got, _ = fa.rotary_forward(x, None, view, rotary, stream=side)
    shared, _ = fa.rotary_forward(x, None, view[:, :1].expand(axes, B, N), rotary)
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert torch.equal(shared[:1], want[:1])
