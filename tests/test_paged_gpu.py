"""Attention over a paged cache, and appending to it, against 64-bit values."""

import math

import pytest
import torch

from paged_plain import BF16, E4M3, Step, angles64, attention64, attention_bounds, turn64

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    from exact_attention_27_gb300 import _build
    _build.build()
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")


def attend(step, causal=True, scale=None, max_q_len=None, stream=None):
    """fa_forward_paged into NaN outputs; the rows past the last sequence must keep them."""
    import exact_attention_27_gb300 as fa
    scale = scale or 1.0 / math.sqrt(step.d)
    cache, batch = step.handles(max_q_len)
    o = torch.full((step.T, step.Hq, step.d), float("nan"), dtype=torch.bfloat16, device="cuda")
    lse = torch.full((step.T, step.Hq), float("nan"), device="cuda")
    ws = fa.paged_workspace(cache, batch, step.q)
    ws.fill_(0xFF)
    fa.fa_forward_paged(cache, batch, step.q, o, lse, scale, causal, ws, stream)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    used = sum(step.q_lens)
    assert torch.isnan(o[used:]).all() and torch.isnan(lse[used:]).all()
    return o, lse, scale


def run(step, causal=True, **kw):
    o, lse, scale = attend(step, causal, **kw)
    step.check(o, lse, scale, causal)
    return o, lse


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("page", [16, 64, 256])
def test_single_tokens(d, e4m3, page):
    lens = [1, 15, 16, 17, 63, 64, 65, 127, 129, 300, 777]
    run(Step([1] * len(lens), lens, 8, 2, d, page, e4m3, seed=d + page, pad=3))


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 96, 128, 256])
@pytest.mark.parametrize("causal", [True, False])
def test_ragged_chunks(d, e4m3, causal):
    """Chunks of every kind in one call: none, one token, a whole prompt, part of one."""
    q = [0, 1, 33, 128, 129, 5, 0, 200]
    k = [40, 700, 33, 128, 400, 6, 0, 513]
    run(Step(q, k, 6, 2, d, 32, e4m3, seed=d + causal, pad=1), causal)


@pytest.mark.parametrize("Hq,Hkv", [(1, 1), (4, 4), (7, 1), (5, 5), (10, 2), (40, 8), (48, 2), (130, 1), (300, 1)])
def test_head_groups(Hq, Hkv):
    run(Step([1, 4, 30], [90, 260, 31], Hq, Hkv, 128, 16, seed=Hq))


@pytest.mark.parametrize("page", [16, 32, 64, 128, 256])
@pytest.mark.parametrize("e4m3", [False, True])
def test_page_sizes(page, e4m3):
    run(Step([1, 70, 2], [page, 3 * page + 1, 2 * page - 1 + 2], 4, 2, 64, page, e4m3, seed=page))


@pytest.mark.parametrize("layout", ["rows", "joint"])
@pytest.mark.parametrize("e4m3", [False, True])
def test_cache_layouts(layout, e4m3):
    run(Step([1, 50], [200, 177], 8, 4, 128, 32, e4m3, seed=3, layout=layout))


@pytest.mark.parametrize("causal", [True, False])
@pytest.mark.parametrize("q_lens", [[3, 0, 1, 9], [3, 0, 1, 90]])
def test_rows_without_keys(causal, q_lens):
    """A length below the number of new tokens leaves the first of them without keys, a length of
    zero all: o = 0, lse = -inf."""
    o, lse = run(Step(q_lens, [0, 5, 0, 4], 4, 2, 64, 16, seed=1), causal)
    assert torch.all(o[:3] == 0) and torch.all(lse[:3] == -math.inf)


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_nan_in_a_query_stays_in_its_row(d, e4m3):
    """o and lse of the row are NaN (not the -infinity of a row without keys), in items that one
    CTA finishes and in items that many join; every other row keeps its bits."""
    for q, k in (([1, 2, 1], [70, 20, 9000]), ([1, 300, 40], [70, 400, 9000])):
        step = Step(q, k, 4, 2, d, 16, e4m3, seed=18)
        o, lse = run(step)
        rows = [(0, 1), (2, 3), (step.T - 1, 0)]
        for t, h in rows:
            step.q[t, h, 5] = float("nan")
        bad_o, bad_lse, _ = attend(step)
        hit = torch.zeros(step.T, 4, dtype=torch.bool, device="cuda")
        for t, h in rows:
            hit[t, h] = True
        assert torch.isnan(bad_o[hit]).all() and torch.isnan(bad_lse[hit]).all()
        assert torch.equal(bad_o[~hit], o[~hit]) and torch.equal(bad_lse[~hit], lse[~hit])


def test_shared_pages():
    """Two sequences with the same beginning, whose pages both read."""
    step = Step([1, 40], [160, 200], 4, 2, 64, 16, seed=15)
    shared = 9
    step.table_cpu[1, :shared] = step.table_cpu[0, :shared]
    step.table = step.table_cpu.cuda()
    step.k64[1][:16 * shared] = step.k64[0][:16 * shared]
    step.v64[1][:16 * shared] = step.v64[0][:16 * shared]
    run(step)


@pytest.mark.parametrize("past", [0, 1, 127, 128, 129, 1000])
@pytest.mark.parametrize("d", [64, 128, 256])
def test_long_chunks(d, past):
    """Items of every length in one sequence, and rows on both sides of a tile's end."""
    for n in (127, 128, 129, 700):
        run(Step([n], [n + past], 2, 1, d, 64, seed=n + past))


@pytest.mark.parametrize("bound", [0, 1, 2, 1000])
def test_wrong_max_q_len_costs_time_only(bound):
    run(Step([1, 20, 90], [50, 40, 300], 4, 1, 64, 16, seed=2), max_q_len=bound)


def test_one_token_over_a_long_history():
    """One key/value head: its keys are divided among all CTAs and joined."""
    run(Step([1], [40001], 4, 1, 64, 64, seed=4))
    run(Step([2, 1], [30000, 7], 5, 1, 128, 64, True, seed=5))


def test_many_sequences():
    """More sequences than a block has threads, most with one key, some without tokens."""
    n = 1100
    q = [i % 3 != 1 and 1 or 0 for i in range(n)]
    k = [1 + (i * 37) % 90 if i % 11 == 0 else 1 for i in range(n)]
    run(Step(q, k, 2, 1, 64, 16, seed=6))
    # ... and with chunks among them
    for i in (0, 5, 500, 777, 1099):
        q[i], k[i] = 30 + i % 7, 40 + i % 90
    run(Step(q, k, 2, 1, 64, 16, seed=6))
    q = [10 + i % 5 for i in range(40)]
    run(Step(q, [n + 7 * i for i, n in enumerate(q)], 4, 1, 256, 16, True, seed=6))


@pytest.mark.parametrize("k_scale", [30.0, 1e-3])
def test_steep_and_flat_scores(k_scale):
    """Scores in the hundreds (one key takes all) and near zero."""
    run(Step([1, 60], [500, 300], 4, 2, 128, 16, seed=7, k_scale=k_scale))
    run(Step([1, 60], [500, 300], 4, 2, 128, 16, True, seed=7, k_scale=min(k_scale, 4.0)))


@pytest.mark.parametrize("q_scale", [1e-30, 1e-6, 1e4])
def test_small_and_large_queries_over_8_bit_keys(q_scale):
    """bf16 queries far outside fp16's range."""
    step = Step([1, 9], [100, 64], 4, 2, 128, 16, True, seed=8)
    step.q_cpu = (step.q_cpu.float() * q_scale).to(torch.bfloat16)
    step.q_cpu[0, 0, 5] = 0.0
    step.q = step.q_cpu.cuda()
    o, lse, scale = attend(step, scale=0.5 / max(q_scale, 1e-6))
    step.check(o, lse, scale, True)


def test_strided_queries_and_outputs():
    """q as a slice of a fused projection, o as a slice of a wider tensor."""
    import exact_attention_27_gb300 as fa
    step = Step([1, 20, 3], [30, 77, 300], 4, 2, 128, 16, seed=9)
    wide = torch.zeros(step.T, 8, 128, dtype=torch.bfloat16, device="cuda")
    wide[:, 2:6] = step.q
    out = torch.zeros(step.T, 9, 128, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(step.T, 4, device="cuda")
    cache, batch = step.handles()
    ws = fa.paged_workspace(cache, batch, step.q)
    fa.fa_forward_paged(cache, batch, wide[:, 2:6], out[:, 5:], lse, 0.1, True, ws)
    torch.cuda.synchronize()
    step.check(out[:, 5:], lse, 0.1, True)
    assert torch.all(out[:, :5] == 0)
    out.zero_()
    fa.fa_forward_paged(cache, batch, wide[:, 2:6], out[:, 5:], None, 0.1, True, ws)
    torch.cuda.synchronize()
    step.check(out[:, 5:], lse, 0.1, True)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("at", [16, 48, 240])
def test_workspace_on_any_16_bytes(d, at):
    """The workspace starts on a 16-byte boundary and no larger one; nothing past its end is
    written."""
    import exact_attention_27_gb300 as fa
    step = Step([1, 300], [5000, 400], 4, 2, d, 16, seed=16)
    cache, batch = step.handles()
    n = fa.paged_workspace(cache, batch, step.q).nbytes
    room = torch.full((n + 512,), 0xA5, dtype=torch.uint8, device="cuda")
    o, lse = torch.empty_like(step.q), torch.empty(step.T, 4, device="cuda")
    fa.fa_forward_paged(cache, batch, step.q, o, lse, 0.1, True, room[at:at + n])
    torch.cuda.synchronize()
    step.check(o, lse, 0.1, True)
    assert torch.all(room[:at] == 0xA5) and torch.all(room[at + n:] == 0xA5)


def test_offsets_past_32_bits():
    """Pages whose elements lie past 2^31."""
    import exact_attention_27_gb300 as fa
    Hkv, page, d = 8, 256, 128
    n_pages = 9000  # 9000 x 8 x 256 x 128 = 2.36e9 elements
    k = torch.zeros(n_pages, Hkv, page, d, dtype=torch.float8_e4m3fn, device="cuda")
    v = torch.zeros_like(k)
    step = Step([1, 40], [300, 511], 16, Hkv, d, page, True, seed=10, spare=0)
    step.table_cpu[step.table_cpu >= 0] += n_pages - step.k_pages.shape[0]
    for small, big in ((step.k_pages, k), (step.v_pages, v)):
        big[n_pages - small.shape[0]:] = small
    step.k_pages, step.v_pages = k, v
    step.table = step.table_cpu.cuda()
    run(step)
    cache, batch = step.handles()
    x = torch.randn(41, Hkv, d, device="cuda").to(torch.bfloat16)
    fa.fa_paged_append(cache, batch, x, x)
    torch.cuda.synchronize()
    last = step.table_cpu[1, 1]
    want = (x[40].float() / step.kd).to(torch.float8_e4m3fn).float()
    assert torch.equal(k[last, :, (511 - 1) % page].float(), want)


def test_bad_pages_and_lengths_are_reported():
    """A page outside the cache, and a length past the table's row, are reported; the other
    sequences have their values, and the device goes on."""
    import exact_attention_27_gb300 as fa
    for what in ("page", "negative", "length"):
        step = Step([1, 1, 40], [100, 200, 90], 4, 2, 64, 16, seed=11)
        if what == "length":
            step.kv_len[1] = 10 ** 9
            # (its row of the table is filled, as its whole length counts)
            step.table[1] = step.table[1].clamp(min=0)
        else:
            step.table[1, 3] = -1 if what == "negative" else 2 ** 31 - 1
        cache, batch = step.handles()
        o, lse = fa.paged_attention(cache, batch, step.q)
        torch.cuda.synchronize()
        assert fa.fa_last_device_error() == fa.FA_ERR_BAD_PAGE, what
        assert fa.fa_last_device_error() == 0
        step.check(o, lse, 1.0 / 8.0, True, only=(0, 2))
        before = step.k_pages.clone().view(torch.int16)
        if what != "length":
            step.table[1, 200 // 16] = step.table[1, 3]
        x = torch.ones(42, 2, 64, dtype=torch.bfloat16, device="cuda")
        fa.fa_paged_append(cache, batch, x, x)
        torch.cuda.synchronize()
        assert fa.fa_last_device_error() == fa.FA_ERR_BAD_PAGE, what
        # only the places of sequences 0 and 2 changed
        changed = (step.k_pages.view(torch.int16) != before).any(-1).any(1).sum().item()
        assert changed == 41
    run(Step([1], [100], 4, 2, 64, 16, seed=12))


def test_nothing_to_do():
    import exact_attention_27_gb300 as fa
    step = Step([0, 0], [5, 0], 4, 2, 64, 16, seed=13, pad=2)
    run(step)
    empty = Step([], [], 4, 2, 64, 16, seed=13)
    cache, batch = empty.handles(1)
    o, lse = fa.paged_attention(cache, batch, empty.q)
    assert o.shape == (0, 4, 64) and lse.shape == (0, 4)
    cache, batch = step.handles(1)
    x = torch.ones(2, 2, 64, dtype=torch.bfloat16, device="cuda")
    before = step.k_pages.clone()
    q = fa.paged_append(cache, batch, x, x, q=step.q)
    torch.cuda.synchronize()
    assert q.shape == step.q.shape
    assert torch.equal(step.k_pages.view(torch.int16), before.view(torch.int16))


def test_same_bits_again():
    step = Step([1, 1, 300, 9], [5000, 70, 900, 2000], 8, 2, 128, 16, seed=14)
    a = attend(step)
    for _ in range(3):
        b = attend(step)
        assert torch.equal(a[0].view(torch.int16), b[0].view(torch.int16))
        assert torch.equal(a[1], b[1])


def test_streams_and_graphs():
    """Two streams at once with a workspace each; a captured call replayed with other lengths,
    pages and values; two graphs in flight."""
    import exact_attention_27_gb300 as fa
    steps = [Step([1, 1, 1], [900, 40, 333], 8, 2, 128, 16, seed=20 + i) for i in range(2)]
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    outs = []
    for _ in range(5):
        for st, s in zip(steps, streams):
            cache, batch = st.handles()
            outs.append((st, fa.paged_attention(cache, batch, st.q, stream=s)))
    torch.cuda.synchronize()
    for st, (o, lse) in outs:
        st.check(o, lse, 1 / math.sqrt(128), True)

    graphs = []
    for st in steps:
        cache, batch = st.handles()
        fa.paged_attention(cache, batch, st.q)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = fa.paged_attention(cache, batch, st.q)
        graphs.append((st, g, out, cache, batch))
    for _ in range(3):
        for (st, g, out, *_), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
    torch.cuda.synchronize()
    for st, g, (o, lse), *_ in graphs:
        st.check(o, lse, 1 / math.sqrt(128), True)
    st, g, (o, lse), *_ = graphs[0]
    st.kv_lens = [700, 33, 1]
    st.k64 = [x[:n] for x, n in zip(st.k64, st.kv_lens)]
    st.v64 = [x[:n] for x, n in zip(st.v64, st.kv_lens)]
    st.kv_len.copy_(torch.tensor(st.kv_lens, dtype=torch.int32))
    st.q_cpu = (st.q_cpu.float() * 0.5).to(torch.bfloat16)
    st.q.copy_(st.q_cpu)
    g.replay()
    torch.cuda.synchronize()
    st.check(o, lse, 1 / math.sqrt(128), True)


# ------------------------------------------------------------------ append


def check_stored(pages, step, new, descale, slack):
    """New rows [T, H, d] (64-bit values) in their places; one rounding and `slack`."""
    pages = pages.cpu().float().double()
    t = 0
    for s, (n, m) in enumerate(zip(step.q_lens, step.kv_lens)):
        for i in range(n):
            j = m - n + i
            if j >= 0:
                got = pages[step.table_cpu[s, j // step.page], :, j % step.page]
                want = new[t + i] / descale
                if step.e4m3:
                    want = want.clamp(-448, 448)
                    tol = E4M3 * want.abs() + 2.0 ** -10
                else:
                    tol = BF16 * want.abs()
                assert torch.all((got - want).abs() <= tol + slack[t + i] / descale + 1e-30)
        t += n


@pytest.mark.parametrize("e4m3", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (96, 96), (96, 32), (128, 128), (128, 64), (256, 256)])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("where", ["place", "text", "video"])
def test_append(d, rot, e4m3, interleaved, where):
    import exact_attention_27_gb300 as fa
    step = Step([3, 0, 1, 40, 2], [3, 9, 70, 55, 0], 4, 2, d, 16, e4m3, seed=d + rot, pad=2,
                layout="rows" if rot == d else "pages")
    cache, batch = step.handles()
    g = torch.Generator().manual_seed(1)
    kv = torch.randn(step.T, 2 * step.Hkv, d, generator=g).to(torch.bfloat16)
    # some values saturate an 8-bit cache
    kv[5, :, 7] = 60.0
    k, v = kv[:, :step.Hkv], kv[:, step.Hkv:]
    inv = (10000.0 ** (-torch.arange(rot // 2, dtype=torch.float64) * 2 / rot)).float()
    axes = 3 if where == "video" else 1
    sections = (rot // 8, rot // 8, rot // 2 - rot // 4) if axes == 3 else None
    axis = torch.tensor([a for a, n in enumerate(sections or (rot // 2,)) for _ in range(n)])
    rotary = fa.Rotary(inv.cuda(), sections, interleaved)
    place = torch.cat([torch.arange(m - n, m) for n, m in zip(step.q_lens, step.kv_lens)] +
                      [torch.zeros(2, dtype=torch.int64)])
    pos = place[None] if where == "place" else \
        torch.randint(0, 10 ** 6, (axes, step.T), generator=g)
    positions = None if where == "place" else pos.to(torch.int32).cuda()
    untouched_k, untouched_v = step.k_pages.clone(), step.v_pages.clone()
    q_out = torch.full(step.q.shape, float("nan"), dtype=torch.bfloat16, device="cuda")
    kv = kv.cuda()
    fa.fa_paged_append(cache, batch, kv[:, :step.Hkv], kv[:, step.Hkv:], rotary, positions, step.q,
                       q_out)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    angle = angles64(pos, inv, axis)[:, None]
    k64, ks = turn64(k.double(), angle, rot, interleaved)
    q64, qs = turn64(step.q_cpu.double(), angle, rot, interleaved)
    used = sum(step.q_lens)
    assert torch.isnan(q_out[used:]).all()
    err = (q_out[:used].cpu().double() - q64[:used]).abs()
    assert torch.all(err <= BF16 * q64[:used].abs() + qs[:used])
    check_stored(step.k_pages, step, k64, step.kd, ks)
    check_stored(step.v_pages, step, v.double(), step.vd, torch.zeros_like(ks))
    # every other place keeps its bits
    keep = torch.ones(step.k_pages.shape[0], step.page, dtype=torch.bool)
    for s, (n, m) in enumerate(zip(step.q_lens, step.kv_lens)):
        for j in range(max(0, m - n), m):
            keep[step.table_cpu[s, j // step.page], j % step.page] = False
    for now, was in ((step.k_pages, untouched_k), (step.v_pages, untouched_v)):
        a, b = (x.transpose(1, 2).contiguous().view(torch.uint8)[keep.cuda()] for x in (now, was))
        assert torch.equal(a, b)


@pytest.mark.parametrize("S", [1, 2, 31, 32, 33, 64, 300])
@pytest.mark.parametrize("pad", [0, 3])
def test_append_finds_every_sequence(S, pad):
    """Around the 32 sequences that a warp holds at once, some without tokens; more key heads
    than a block goes through at a time."""
    import exact_attention_27_gb300 as fa
    q = [(5 * i + 2) % 4 for i in range(S)]
    step = Step(q, [n + (7 * i) % 50 for i, n in enumerate(q)], 24, 24, 64, 16, seed=S, pad=pad)
    cache, batch = step.handles()
    k, v = (torch.randn(step.T, 24, 64, device="cuda").to(torch.bfloat16) for _ in range(2))
    fa.fa_paged_append(cache, batch, k, v)
    torch.cuda.synchronize()
    assert fa.fa_last_device_error() == 0
    none = torch.zeros(step.T, 24, 64)
    check_stored(step.k_pages, step, k.cpu().double(), 1.0, none)
    check_stored(step.v_pages, step, v.cpu().double(), 1.0, none)


def test_append_turns_q_in_place():
    import exact_attention_27_gb300 as fa
    step = Step([5, 2], [5, 90], 4, 2, 64, 16, seed=3)
    cache, batch = step.handles()
    k = torch.randn(7, 2, 64, device="cuda").to(torch.bfloat16)
    inv = (10000.0 ** (-torch.arange(32, dtype=torch.float64) / 32)).float()
    rotary = fa.Rotary(inv.cuda())
    want = fa.paged_append(cache, batch, k, k, rotary, q=step.q)
    fa.fa_paged_append(cache, batch, k, k, rotary, None, step.q, step.q)
    torch.cuda.synchronize()
    assert torch.equal(step.q, want)


def test_append_without_rotation_copies():
    import exact_attention_27_gb300 as fa
    step = Step([4, 1], [4, 33], 4, 2, 128, 16, seed=2)
    cache, batch = step.handles()
    k = torch.randn(5, 2, 128, device="cuda").to(torch.bfloat16)
    one = torch.randn(5, 1, 128, device="cuda").to(torch.bfloat16)
    fa.fa_paged_append(cache, batch, k, one.expand(5, 2, 128))
    torch.cuda.synchronize()
    check_stored(step.k_pages, step, k.cpu().double(), 1.0, torch.zeros(5, 2, 128))
    check_stored(step.v_pages, step, one.expand(5, 2, 128).cpu().double(), 1.0,
                 torch.zeros(5, 2, 128))


@pytest.mark.parametrize("e4m3", [False, True])
def test_serving_steps_equal_dense_attention(e4m3):
    """Prompts in chunks, then tokens one by one, through append and attention: each step's
    output is attention over everything appended so far."""
    import exact_attention_27_gb300 as fa
    d, Hq, Hkv, page, S = 128, 8, 2, 16, 3
    total = [150, 97, 40]
    g = torch.Generator().manual_seed(5)
    data = [tuple(torch.randn(n, h, d, generator=g).to(torch.bfloat16) for h in (Hq, Hkv, Hkv))
            for n in total]
    dtype = torch.float8_e4m3fn if e4m3 else torch.bfloat16
    kd, vd = (0.125, 0.0625) if e4m3 else (1.0, 1.0)
    pages = [torch.full((40, Hkv, page, d), float("nan"), device="cuda").to(dtype)
             for _ in range(2)]
    cache = fa.PagedCache(pages[0], pages[1], kd, vd)
    table = torch.randperm(40, generator=g)[:30].view(S, 10).to(torch.int32).cuda()
    inv = (10000.0 ** (-torch.arange(64, dtype=torch.float64) / 64)).float()
    rotary = fa.Rotary(inv.cuda())
    done = [0] * S
    q64, k64, v64 = [], [], []
    for s in range(S):
        angle = angles64(torch.arange(total[s])[None], inv, torch.zeros(64))[:, None]
        q64.append(turn64(data[s][0].double(), angle, d, False)[0].float().to(
            torch.bfloat16).double())
        k = turn64(data[s][1].double(), angle, d, False)[0]
        k64.append((k / kd).float().to(dtype).double() * kd)
        v64.append((data[s][2].double() / vd).float().to(dtype).double() * vd)
    steps = [[70, 0, 40], [1, 90, 0], [64, 1, 0]] + [[1, 1, 0]] * 5 + [[10, 1, 0]]
    for new in steps:
        take = [tuple(x[a:a + n] for x in data[s]) for s, (a, n) in enumerate(zip(done, new))]
        done = [a + n for a, n in zip(done, new)]
        q, k, v = (torch.cat([t[i] for t in take]).cuda() for i in range(3))
        starts = torch.tensor([sum(new[:i]) for i in range(S + 1)], dtype=torch.int32).cuda()
        batch = fa.PagedBatch(table, starts, torch.tensor(done, dtype=torch.int32).cuda(),
                              max(new))
        q = fa.paged_append(cache, batch, k, v, rotary, q=q)
        o, lse = fa.paged_attention(cache, batch, q)
        torch.cuda.synchronize()
        assert fa.fa_last_device_error() == 0
        at = 0
        for s, n in enumerate(new):
            if n:
                m = done[s]
                ro, rl, a, size = attention64(q64[s][m - n:m], k64[s][:m], v64[s][:m],
                                              1 / math.sqrt(d), True, m - n)
                ot, lt = attention_bounds(ro, rl, a, size, d, m, v64[s].abs().max().item(), e4m3)
                # q and k were rounded from fp32 values within 2^-20 of the 64-bit ones: now and
                # then to the neighbouring value, a step (2^-7, or 2^-3 for e4m3) of one of d
                # products; four of them at once are allowed for
                step = (2.0 ** -3 if e4m3 else 2.0 ** -7) * 4 * 9.0 / math.sqrt(d)
                err = (o[at:at + n].cpu().double() - ro).abs()
                assert torch.all(err <= ot + step * 2 * a)
                assert torch.all((lse[at:at + n].cpu().double() - rl).abs() <= lt + step)
            at += n
    # bf16: the same as the dense forward on what was appended
    if not e4m3:
        s, m = 0, done[0]
        dense = [x[s][:m].transpose(0, 1)[None].to(torch.bfloat16).cuda().contiguous()
                 for x in (q64, k64, v64)]
        o2, _ = fa.attention_forward(*dense, causal=True)
        diff = (o2[0].transpose(0, 1)[m - 10:m].float() - o[:10].float()).abs()
        assert diff.max() <= 2e-2
