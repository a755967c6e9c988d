"""Refusals of the rotary and paged entry points: on the host, before any CUDA call."""

import ctypes

import pytest
import torch

import exact_attention_27_gb300 as fa
from exact_attention_27_gb300 import _build, _lib

# Fake, 16-byte aligned, never dereferenced: validation fails before any use.
P = 0x10000
Q = 0x10008  # 8-byte aligned only
F = 0x10002  # 2-byte aligned only


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return fa.library()


def spec(**kw):
    a = dict(inv_freq=P, rot_dim=64, axes=2, interleaved=0)
    axis = kw.pop("axis", [0] * 16 + [1] * 16)
    a.update(kw)
    return _lib.RotarySpec(a["inv_freq"], a["rot_dim"], a["axes"], a["interleaved"],
                           (ctypes.c_ubyte * 128)(*axis))


def rows(**kw):
    a = dict(in_=P, out=P, in_batch=4096, in_head=512, in_pos=64, out_batch=4096, out_head=512,
             out_pos=64, heads=2)
    a.update(kw)
    return _lib.RotaryRows(**a)


def rotary(lib, fn="fa_rotary", q=None, k=None, B=2, N=8, d=64, pos=P, axis=16, batch=8, s=None):
    ref = ctypes.byref
    q = rows() if q is None else q
    return getattr(lib, fn)(ref(q) if q else None, ref(k) if k else None, B, N, d, pos, axis,
                            batch, ref(spec() if s is None else s), None)


@pytest.mark.parametrize("fn", ["fa_rotary", "fa_rotary_backward"])
@pytest.mark.parametrize("kw", [
    dict(q=False), dict(B=0), dict(N=0), dict(N=-1), dict(pos=None), dict(pos=F), dict(axis=-1),
    dict(batch=-8), dict(q=rows(in_=None)), dict(q=rows(out=Q)), dict(q=rows(heads=0)),
    dict(q=rows(in_pos=60)), dict(q=rows(in_head=-64)), dict(q=rows(out_pos=0)),
    dict(q=rows(out_head=0)), dict(q=rows(out_batch=4)), dict(k=rows(heads=0)),
    dict(k=rows(in_=Q)), dict(B=2 ** 20, N=2 ** 20), dict(q=rows(heads=2 ** 20)),
    dict(s=spec(inv_freq=None)), dict(s=spec(rot_dim=0)), dict(s=spec(rot_dim=24)),
    dict(s=spec(rot_dim=80)), dict(s=spec(axes=0)), dict(s=spec(axes=5)), dict(s=spec(axes=1)),
    dict(s=spec(interleaved=2)), dict(s=spec(axis=[0] * 31 + [2])),
])
def test_rotary_rejects(lib, fn, kw):
    assert rotary(lib, fn, **kw) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("d", [0, 32, 80, 512])
def test_rotary_rejects_unsupported_head_dim(lib, d):
    assert rotary(lib, d=d) == fa.FA_ERR_UNSUPPORTED
    assert append(lib, c=cache(d=d)) == fa.FA_ERR_UNSUPPORTED
    assert forward(lib, c=cache(d=d)) == fa.FA_ERR_UNSUPPORTED


def cache(**kw):
    a = dict(k=P, v=P, page_stride=2048, head_stride=1024, row_stride=64, n_pages=4, page_size=16,
             H_kv=2, d=64, dtype=0, k_descale=1.0, v_descale=1.0)
    a.update(kw)
    return _lib.PagedCacheStruct(**a)


def batch(**kw):
    a = dict(block_table=P, table_stride=4, max_pages=4, q_start=P, kv_len=P, S=2, max_q_len=1)
    a.update(kw)
    return _lib.PagedBatchStruct(**a)


def append(lib, c=None, b=None, **kw):
    a = dict(k=P, kt=128, kh=64, v=P, vt=128, vh=64, T=2, q=P, qt=256, qh=64, o=P, ot=256, oh=64,
             Hq=4, s=None, pos=None, axis=0)
    a.update(kw)
    ref = ctypes.byref
    return lib.fa_paged_append(
        ref(c or cache()), ref(b or batch()), a["k"], a["kt"], a["kh"], a["v"], a["vt"], a["vh"],
        a["T"], a["q"], a["qt"], a["qh"], a["o"], a["ot"], a["oh"], a["Hq"],
        None if a["s"] is None else ref(a["s"]), a["pos"], a["axis"], None)


def forward(lib, c=None, b=None, **kw):
    a = dict(q=P, qt=256, qh=64, o=P, ot=256, oh=64, lse=P, T=2, Hq=4, scale=0.125, causal=1,
             ws=P, bytes=2 ** 40)
    a.update(kw)
    ref = ctypes.byref
    return lib.fa_forward_paged(
        ref(c or cache()), ref(b or batch()), a["q"], a["qt"], a["qh"], a["o"], a["ot"], a["oh"],
        a["lse"], a["T"], a["Hq"], ctypes.c_float(a["scale"]), a["causal"], a["ws"], a["bytes"],
        None)


BAD_CACHES = [dict(k=None), dict(v=Q), dict(n_pages=0), dict(page_size=8), dict(page_size=48),
              dict(page_size=512), dict(H_kv=0), dict(dtype=2), dict(dtype=-1),
              dict(k_descale=0.5), dict(v_descale=2.0), dict(dtype=1, k_descale=0.0),
              dict(dtype=1, v_descale=float("nan")), dict(dtype=1, k_descale=float("inf")),
              dict(row_stride=68), dict(row_stride=32), dict(head_stride=0),
              dict(page_stride=2 ** 39), dict(dtype=1, row_stride=72)]
BAD_BATCHES = [dict(S=-1), dict(max_pages=-1), dict(max_pages=0), dict(max_pages=2 ** 30),
               dict(max_q_len=-1), dict(q_start=None), dict(kv_len=None), dict(block_table=None),
               dict(table_stride=-4), dict(q_start=F), dict(kv_len=F), dict(block_table=F)]


@pytest.mark.parametrize("call", [append, forward])
@pytest.mark.parametrize("kw", BAD_CACHES)
def test_bad_caches_are_rejected(lib, call, kw):
    assert call(lib, c=cache(**kw)) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("call", [append, forward])
@pytest.mark.parametrize("kw", BAD_BATCHES)
def test_bad_batches_are_rejected(lib, call, kw):
    assert call(lib, b=batch(**kw)) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("call", [append, forward])
@pytest.mark.parametrize("kw", [dict(k_descale=1e-39), dict(v_descale=2.0 ** -149)])
def test_descales_without_a_reciprocal_are_rejected(lib, call, kw):
    assert call(lib, c=cache(dtype=1, **kw)) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(k=None), dict(v=None), dict(k=Q), dict(v=Q), dict(T=-1), dict(kt=60), dict(vh=-64),
    dict(q=None), dict(o=None), dict(q=Q), dict(o=Q), dict(Hq=0), dict(qt=4), dict(ot=0),
    dict(oh=0), dict(pos=F), dict(axis=-1), dict(Hq=2 ** 20), dict(s=spec(rot_dim=128)),
    dict(s=spec(rot_dim=8)), dict(s=spec(axis=[3] * 32)),
])
def test_append_rejects(lib, kw):
    assert append(lib, **kw) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [
    dict(q=None), dict(o=None), dict(q=Q), dict(o=Q), dict(lse=F), dict(T=-1), dict(Hq=3),
    dict(Hq=0), dict(scale=0.0), dict(scale=-1.0), dict(scale=float("nan")),
    dict(scale=float("inf")), dict(scale=3e38), dict(causal=2), dict(qt=4), dict(qh=-64), dict(ot=0), dict(oh=0),
    dict(T=2 ** 30, Hq=4),
])
def test_forward_rejects(lib, kw):
    assert forward(lib, **kw) == fa.FA_ERR_INVALID_ARGUMENT


@pytest.mark.parametrize("kw", [dict(T=0), dict(b=batch(S=0))])
def test_nothing_to_do_needs_no_gpu(lib, kw):
    """T = 0 or S = 0 returns FA_OK without pointers or launches."""
    kw = dict(kw)
    b = kw.pop("b", batch(S=2, q_start=None, kv_len=None, block_table=None))
    assert append(lib, c=cache(k=None, v=None), b=b, k=None, v=None, **kw) == fa.FA_OK
    assert forward(lib, c=cache(k=None, v=None), b=b, q=None, o=None, ws=None, **kw) == fa.FA_OK


@pytest.mark.parametrize("args", [(4, 3, 64, 1, 1), (0, 1, 64, 1, 1), (4, 0, 64, 1, 1),
                                  (4, 2, 80, 1, 1), (4, 2, 64, -1, 1), (4, 2, 64, 1, -1)])
def test_workspace_rejects(lib, args):
    assert lib.fa_forward_paged_workspace_bytes(*args) == 0


def test_handles_check_their_tensors():
    x = torch.zeros(4, 2, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        fa.PagedCache(x, x)  # not on the GPU
    with pytest.raises(ValueError):
        fa.PagedCache(x, x[:3])
    with pytest.raises(ValueError):
        fa.PagedCache(x.half(), x.half())
    with pytest.raises(ValueError):
        fa.Rotary(torch.zeros(32))
    i = torch.zeros(2, 4, dtype=torch.int32)
    with pytest.raises(ValueError):
        fa.PagedBatch(i, torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float8_e4m3fn])
@pytest.mark.parametrize("broadcast", [0, 1, 2])
def test_broadcast_pages_are_refused(dtype, broadcast):
    """Pages, heads or rows that share their memory: a view with a stride of 0."""
    shape = [4, 2, 16, 64]
    one = list(shape)
    one[broadcast] = 1
    x = torch.zeros(one, dtype=torch.float32).to(dtype).expand(shape)
    with pytest.raises(ValueError, match="strides"):
        fa.PagedCache(x, x)


def test_rows_as_bytes_are_the_struct():
    from exact_attention_27_gb300 import paged
    values = (1 << 40, 2 << 40, 3, 4, 5 << 33, 6, 7, 8, 9)
    assert paged._rows_bytes(*values) == bytes(_lib.RotaryRows(*values))


def test_status_of_a_bad_page(lib):
    assert "page" in fa.fa_status_string(fa.FA_ERR_BAD_PAGE)
