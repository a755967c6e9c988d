"""Binding of the rotary-position and paged-cache entry points of include/fa.h.

What a program keeps for many calls is checked once, in a handle that holds its
tensors and mirrors a struct of the C interface: `Rotary` (of a model),
`PagedCache` (of a layer) and `PagedBatch` (of a step, shared by its layers).
The handles hold addresses, not values: a tensor written in place is seen by the
next call, and a captured graph replays with what the tensors then hold.

The fa_* functions write into the caller's tensors; rotary_forward,
rotary_backward, paged_append and paged_attention allocate what they return.
"""

import ctypes
import math
import struct

from . import _lib
from ._lib import FaError, library

_byref = ctypes.byref
# An fa_rotary_rows as bytes, which a call takes for a pointer (a third of the time of filling a
# ctypes structure).
_rows_bytes = struct.Struct("PPqqqqqqi4x").pack

# torch is imported on first use, by the first handle; what every call asks for is then at hand
# (a server's step makes two calls a layer, and each microsecond of host time counts there).
_torch = _BF16 = _F32 = _I32 = _contiguous = None
_device = _raw_stream = None


def _load_torch():
    global _torch, _BF16, _F32, _I32, _contiguous, _device, _raw_stream
    if _torch is None:
        import torch
        _BF16, _F32, _I32 = torch.bfloat16, torch.float32, torch.int32
        _contiguous = torch.contiguous_format
        _device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
            lambda _: torch.cuda.current_stream().cuda_stream)
        _torch = torch
    return _torch


def _stream(stream, device):
    if stream is None:
        return _raw_stream(device)
    return stream if isinstance(stream, int) else stream.cuda_stream


def _on(stream):
    """Allocations on `stream`, whose later use on it the allocator then orders."""
    if isinstance(stream, int):
        stream = _torch.cuda.ExternalStream(stream)
    return _torch.cuda.stream(stream)


def _int32(name, t, dims, device=None):
    if not isinstance(t, _torch.Tensor) or t.dtype is not _I32 or not t.is_cuda:
        raise ValueError(f"{name} must be an int32 CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimension(s), has {t.dim()}")
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError(f"{name} must be contiguous along its last dimension")
    if device is not None and t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not cuda:{device}")


def _rows3(name, t, device):
    """Token and head strides of a bf16 [T, heads, d] on `device`, its last dimension
    contiguous; the library checks the address."""
    s = t.stride()
    if t.dtype is _BF16 and t.get_device() == device and len(s) == 3 and s[2] == 1 and \
            not (s[0] | s[1]) & 7:
        return s
    return _strides(name, t, 3, device)


def _strides(name, t, dims, device):
    """The strides of a bf16 CUDA tensor of `dims` dimensions addressed in 16-byte vectors (those
    of dimensions of one element, which may be anything, rounded to what the library takes)."""
    if t.dtype is not _BF16 or not t.is_cuda:
        raise ValueError(f"{name} must be a bf16 CUDA tensor")
    if t.dim() != dims:
        raise ValueError(f"{name} must have {dims} dimensions, has {t.dim()}")
    if t.get_device() != device:
        raise ValueError(f"{name} is on cuda:{t.get_device()}, not cuda:{device}")
    strides = t.stride()
    if strides[-1] != 1:
        raise ValueError(f"{name} must be contiguous along d")
    for n, s in zip(t.shape, strides[:-1]):
        if s & 7 and n > 1:
            raise ValueError(f"{name} has strides {strides}: multiples of 8 are needed")
    return tuple((s + 7) & ~7 for s in strides)


def _same_device(device, *handles):
    for h in handles:
        if h is not None and h.device != device:
            raise ValueError(f"{type(h).__name__} is on cuda:{h.device}, the tensors on "
                             f"cuda:{device}")
    if device != _device():
        raise ValueError(f"the tensors are on cuda:{device}, the current device is "
                         f"cuda:{_device()}")


class Rotary:
    """Rotary positions of a model: inv_freq [rot_dim / 2] fp32 (radians a position, on the
    GPU); `sections` how many consecutive pairs each axis turns ((rot_dim / 2,) for text), or
    `axis_of_pair` the axis of every pair; `interleaved` pairs (2p, 2p + 1) instead of
    (p, p + rot_dim / 2)."""

    def __init__(self, inv_freq, sections=None, interleaved=False, axis_of_pair=None):
        torch = _load_torch()
        if inv_freq.dtype is not torch.float32 or not inv_freq.is_cuda or inv_freq.dim() != 1 or \
                not inv_freq.is_contiguous():
            raise ValueError("inv_freq must be a contiguous fp32 CUDA vector")
        half = inv_freq.shape[0]
        if half % 8 or not 8 <= half <= 128:
            raise ValueError(f"inv_freq has {half} values: a multiple of 8, 8 to 128, is needed")
        if axis_of_pair is None:
            sections = (half,) if sections is None else tuple(int(n) for n in sections)
            if min(sections, default=-1) < 0 or sum(sections) != half:
                raise ValueError(f"sections {sections} do not add up to {half} pairs")
            axis_of_pair = [a for a, n in enumerate(sections) for _ in range(n)]
            axes = len(sections)
        else:
            if sections is not None:
                raise ValueError("give sections or axis_of_pair, not both")
            axis_of_pair = [int(a) for a in axis_of_pair]
            if len(axis_of_pair) != half or min(axis_of_pair) < 0:
                raise ValueError(f"axis_of_pair must name an axis for each of {half} pairs")
            axes = max(axis_of_pair) + 1
        if not 1 <= axes <= 4:
            raise ValueError(f"{axes} axes: 1 to 4 are supported")
        self.inv_freq, self.axes, self.device = inv_freq, axes, inv_freq.get_device()
        self.rot_dim = 2 * half
        self._c = _lib.RotarySpec(inv_freq.data_ptr(), 2 * half, axes, int(bool(interleaved)),
                                  (ctypes.c_ubyte * 128)(*axis_of_pair))
        self._ref = _byref(self._c)


class PagedCache:
    """One layer's keys and values in pages: k_pages and v_pages [n_pages, H_kv, page_size, d],
    bf16 or float8_e4m3fn (values times the descales), both with the same strides (a permuted
    view of [n_pages, page_size, H_kv, d], or slices of one tensor, will do)."""

    def __init__(self, k_pages, v_pages, k_descale=1.0, v_descale=1.0):
        torch = _load_torch()
        if k_pages.dim() != 4 or k_pages.shape != v_pages.shape:
            raise ValueError("k_pages and v_pages must both be [n_pages, H_kv, page_size, d]")
        kinds = {torch.bfloat16: (0, 2), torch.float8_e4m3fn: (1, 1)}
        if k_pages.dtype not in kinds or v_pages.dtype is not k_pages.dtype:
            raise ValueError("k_pages and v_pages must both be bf16 or both float8_e4m3fn")
        dtype, size = kinds[k_pages.dtype]
        n, H, page, d = k_pages.shape
        if d not in (64, 96, 128, 256):
            raise FaError(2, "PagedCache")
        if page not in (16, 32, 64, 128, 256):
            raise ValueError(f"pages of {page} positions: 16, 32, 64, 128 or 256 are supported")
        if n < 1 or H < 1:
            raise ValueError("the cache is empty")
        for t in (k_pages, v_pages):
            if t.stride(3) != 1 or t.data_ptr() & 15:
                raise ValueError("pages must be contiguous along d and start on 16 bytes")
        # the stride of a dimension of one element is free: use the dense one
        ks, vs = ([t.stride(i) if t.shape[i] > 1 else d * page * H for i in range(3)]
                  for t in (k_pages, v_pages))
        if ks != vs:
            raise ValueError("k_pages and v_pages must have the same strides")
        if any(s * size % 16 or s < d for s in ks):
            raise ValueError(f"page strides {tuple(ks)}: multiples of 16 bytes, at least d, "
                             "are needed")
        if not k_pages.is_cuda or k_pages.get_device() != v_pages.get_device():
            raise ValueError("k_pages and v_pages must be CUDA tensors of one device")
        if not (math.isfinite(k_descale) and k_descale > 0 and math.isfinite(v_descale) and
                v_descale > 0) or (dtype == 0 and (k_descale, v_descale) != (1.0, 1.0)):
            raise ValueError("descales must be finite and > 0, and 1 for bf16 pages")
        self.k_pages, self.v_pages = k_pages, v_pages
        self.n_pages, self.H_kv, self.page_size, self.d = n, H, page, d
        self.device = k_pages.get_device()
        self._c = _lib.PagedCacheStruct(k_pages.data_ptr(), v_pages.data_ptr(), ks[0], ks[1],
                                        ks[2], n, page, H, d, dtype, k_descale, v_descale)
        self._ref = _byref(self._c)


class PagedBatch:
    """One step's sequences: block_table [S, max_pages], q_start [S + 1] and kv_len [S], int32
    on the GPU (fa_paged_batch in include/fa.h).  max_q_len, the most new tokens that one
    sequence brings, chooses kernels; a wrong value costs time only."""

    def __init__(self, block_table, q_start, kv_len, max_q_len=1):
        _load_torch()
        _int32("block_table", block_table, 2)
        device = block_table.get_device()
        _int32("q_start", q_start, 1, device)
        _int32("kv_len", kv_len, 1, device)
        S = kv_len.shape[0]
        if q_start.shape[0] != S + 1 or block_table.shape[0] != S:
            raise ValueError(f"q_start must hold {S + 1} values and block_table {S} rows, as "
                             f"kv_len holds {S}")
        if S and block_table.shape[1] < 1:
            raise ValueError("block_table has no columns")
        self.block_table, self.q_start, self.kv_len = block_table, q_start, kv_len
        self.S, self.max_q_len, self.device = S, int(max_q_len), device
        if self.max_q_len < 0:
            raise ValueError("max_q_len is negative")
        self._c = _lib.PagedBatchStruct(
            block_table.data_ptr(), block_table.stride(0) if S > 1 else block_table.shape[1],
            block_table.shape[1], q_start.data_ptr(), kv_len.data_ptr(), S,
            min(self.max_q_len, 2**31 - 1))
        self._ref = _byref(self._c)


def _rotary_rows(x, out, device, name):
    a, b = x.stride(), out.stride()
    shape = x.shape
    if out.shape != shape:
        raise ValueError(f"{name}_out has shape {tuple(out.shape)}, expected {tuple(shape)}")
    if x.dtype is not _BF16 or out.dtype is not _BF16 or x.get_device() != device or \
            out.get_device() != device or len(a) != 4 or a[3] != 1 or b[3] != 1 or \
            (a[0] | a[1] | a[2] | b[0] | b[1] | b[2]) & 7 or not (b[0] and b[1] and b[2]):
        a = _strides(name, x, 4, device)
        b = _strides(name + "_out", out, 4, device)
        if any(n > 1 and s == 0 for n, s in zip(shape, b)):
            raise ValueError(f"{name}_out is a broadcast view")
    return _rows_bytes(x.data_ptr(), out.data_ptr(), a[0], a[1], a[2], b[0], b[1], b[2], shape[1])


def _launch_turn(fn, rows_q, rows_k, shape, k, positions, rotary, stream):
    B, _, N, d = shape
    device = rotary.device
    if k is not None:
        Bk, _, Nk, dk = k.shape
        if Bk != B or Nk != N or dk != d:
            raise ValueError("k must be [B, H_kv, N, d] with q's B, N and d")
    if device != _device():
        _same_device(device)
    if positions.dim() == 2:
        positions = positions[None]
    s = positions.stride()
    if positions.dtype is not _I32 or positions.get_device() != device or len(s) != 3 or \
            s[2] != 1:
        _int32("positions", positions, 3, device)
    if positions.shape != (rotary.axes, B, N):
        raise ValueError(f"positions have shape {tuple(positions.shape)}, expected "
                         f"{(rotary.axes, B, N)}")
    status = getattr(library(), fn)(rows_q, rows_k, B, N, d, positions.data_ptr(), s[0],
                                    s[1], rotary._ref, _stream(stream, device))
    if status:
        raise FaError(status, fn)


def _turn(fn, q, q_out, k, k_out, positions, rotary, stream):
    if (k is None) != (k_out is None):
        raise ValueError("give k and its output, or neither")
    device = rotary.device
    _launch_turn(fn, _rotary_rows(q, q_out, device, "q"),
                 None if k is None else _rotary_rows(k, k_out, device, "k"), q.shape, k, positions,
                 rotary, stream)


def fa_rotary(q, q_out, k, k_out, positions, rotary, stream=None):
    """fa_rotary of include/fa.h on torch tensors: q [B, H_q, N, d] (and k [B, H_kv, N, d], or
    None) bf16 views turned into q_out and k_out, which may be q and k; positions
    [axes, B, N] int32, or [B, N] for one axis (expanded views share rows)."""
    _turn("fa_rotary", q, q_out, k, k_out, positions, rotary, stream)


def fa_rotary_backward(dq_out, dq, dk_out, dk, positions, rotary, stream=None):
    """fa_rotary_backward of include/fa.h: gradients of fa_rotary's outputs turned back into
    gradients of its inputs."""
    _turn("fa_rotary_backward", dq_out, dq, dk_out, dk, positions, rotary, stream)


def rotary_forward(q, k, positions, rotary, stream=None):
    """Allocates and returns q and k (None: only q) turned by their positions, contiguous (what
    attention_forward takes)."""
    return _new_turn("fa_rotary", q, k, positions, rotary, stream)


def rotary_backward(dq, dk, positions, rotary, stream=None):
    """Gradients of rotary_forward's inputs from those of its outputs (for instance what
    attention_backward returns)."""
    return _new_turn("fa_rotary_backward", dq, dk, positions, rotary, stream)


def _new_rows(x, device, name):
    """A contiguous output for x, and the rows of both."""
    shape, a = x.shape, x.stride()
    if x.dtype is not _BF16 or x.get_device() != device or len(a) != 4 or a[3] != 1 or \
            (a[0] | a[1] | a[2]) & 7:
        a = _strides(name, x, 4, device)
    # (quicker than empty with a type and a device)
    out = _torch.empty_like(x, memory_format=_contiguous)
    _, H, N, d = shape
    return out, _rows_bytes(x.data_ptr(), out.data_ptr(), a[0], a[1], a[2], H * N * d, N * d, d, H)


def _new_turn(fn, q, k, positions, rotary, stream):
    if stream is not None:
        with _on(stream):
            return _new_turn_here(fn, q, k, positions, rotary, stream)
    return _new_turn_here(fn, q, k, positions, rotary, None)


def _new_turn_here(fn, q, k, positions, rotary, stream):
    device = rotary.device
    q_out, rows_q = _new_rows(q, device, "q")
    k_out = rows_k = None
    if k is not None:
        k_out, rows_k = _new_rows(k, device, "k")
    _launch_turn(fn, rows_q, rows_k, q.shape, k, positions, rotary, stream)
    return q_out, k_out


def fa_paged_append(cache, batch, k, v, rotary=None, positions=None, q=None, q_out=None,
                    stream=None):
    """fa_paged_append of include/fa.h: stores the step's k and v [T, H_kv, d] (bf16 views) in
    the cache, k turned by `rotary` at `positions` ([axes, T] int32, or [T] for one axis; None:
    each token's place in its sequence), and writes q [T, H_q, d] turned likewise to q_out."""
    device = cache.device
    ks = _rows3("k", k, device)
    vs = _rows3("v", v, device)
    T, H, d = shape = k.shape
    if v.shape != shape or H != cache.H_kv or d != cache.d:
        raise ValueError(f"k and v must be [T, {cache.H_kv}, {cache.d}]")
    if batch.device != device or device != _device() or \
            (rotary is not None and rotary.device != device):
        _same_device(device, batch, rotary)
    qp = op = None
    q_token = q_head = o_token = o_head = Hq = 0
    if q is not None and q_out is not None:
        q_token, q_head, _ = _rows3("q", q, device)
        o_token, o_head, _ = _rows3("q_out", q_out, device)
        Tq, Hq, dq = q_shape = q.shape
        if Tq != T or dq != d or q_out.shape != q_shape:
            raise ValueError(f"q and q_out must be [{T}, H_q, {d}]")
        qp, op = q.data_ptr(), q_out.data_ptr()
    elif q is not None or q_out is not None:
        raise ValueError("give q and q_out, or neither")
    pp, axis_stride, ref = None, 0, None
    if rotary is not None:
        ref = rotary._ref
        if rotary.rot_dim > d:
            raise ValueError(f"rotary turns {rotary.rot_dim} values of {d}")
    if positions is not None:
        if rotary is None:
            raise ValueError("positions without rotary")
        if positions.dim() == 1:
            positions = positions[None]
        s = positions.stride()
        if positions.dtype is not _I32 or positions.get_device() != device or len(s) != 2 or \
                s[1] != 1:
            _int32("positions", positions, 2, device)
        if positions.shape != (rotary.axes, T):
            raise ValueError(f"positions have shape {tuple(positions.shape)}, expected "
                             f"{(rotary.axes, T)}")
        pp, axis_stride = positions.data_ptr(), s[0]
    if T == 0 or batch.S == 0:
        return
    status = library().fa_paged_append(
        cache._ref, batch._ref, k.data_ptr(), ks[0], ks[1], v.data_ptr(), vs[0], vs[1], T, qp,
        q_token, q_head, op, o_token, o_head, Hq, ref, pp, axis_stride, _stream(stream, device))
    if status:
        raise FaError(status, "fa_paged_append")


def paged_append(cache, batch, k, v, rotary=None, positions=None, q=None, stream=None):
    """fa_paged_append with a q_out of its own, which it returns (None without q).  Rows past
    the last sequence are left as the allocation has them."""
    q_out = None
    if q is not None:
        if stream is not None:
            with _on(stream):
                q_out = _torch.empty(q.shape, dtype=q.dtype, device=q.device)
        else:
            q_out = _torch.empty(q.shape, dtype=q.dtype, device=q.device)
    fa_paged_append(cache, batch, k, v, rotary, positions, q, q_out, stream)
    return q_out


def paged_workspace(cache, batch, q):
    """A workspace for fa_forward_paged calls of this shape.  Its contents do not matter, and
    calls on one stream may share it; calls that can overlap, such as two captured graphs,
    may not."""
    if q.dim() != 3 or q.shape[1] % cache.H_kv or q.shape[1] < 1:
        raise ValueError(f"q must be [T, H_q, {cache.d}] with H_q a multiple of {cache.H_kv}")
    n = library().fa_forward_paged_workspace_bytes(q.shape[1], cache.H_kv, cache.d, q.shape[0],
                                                   batch._c.max_q_len)
    return _torch.empty(n, dtype=_torch.uint8, device=q.device)


def fa_forward_paged(cache, batch, q, o, lse, scale, causal, workspace, stream=None):
    """fa_forward_paged of include/fa.h: the step's q [T, H_q, d] (a bf16 view) against the
    cache; writes o (like q) and lse [T, H_q] fp32 (None: not wanted)."""
    device = cache.device
    q_token, q_head, _ = _rows3("q", q, device)
    o_token, o_head, _ = _rows3("o", o, device)
    T, Hq, d = shape = q.shape
    if d != cache.d or o.shape != shape or Hq < 1 or Hq % cache.H_kv:
        raise ValueError(f"q and o must be [T, H_q, {cache.d}] with H_q a multiple of "
                         f"{cache.H_kv}")
    if batch.device != device or device != _device():
        _same_device(device, batch)
    lp = None
    if lse is not None:
        if lse.dtype is not _F32 or lse.get_device() != device or lse.shape != shape[:2] or \
                not lse.is_contiguous():
            raise ValueError(f"lse must be a contiguous fp32 CUDA tensor [{T}, {Hq}]")
        lp = lse.data_ptr()
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError("workspace must be a contiguous CUDA tensor of the cache's device")
    if T == 0 or batch.S == 0:
        return
    status = library().fa_forward_paged(
        cache._ref, batch._ref, q.data_ptr(), q_token, q_head, o.data_ptr(), o_token, o_head, lp,
        T, Hq, scale, 1 if causal else 0, workspace.data_ptr(), workspace.nbytes,
        _stream(stream, device))
    if status:
        raise FaError(status, "fa_forward_paged")


def paged_attention(cache, batch, q, causal=True, scale=None, stream=None):
    """Allocates o, lse and the workspace and runs fa_forward_paged; returns (o, lse).  Rows
    past the last sequence are left as the allocations have them."""
    if stream is not None:
        with _on(stream):
            return _paged_attention(cache, batch, q, causal, scale, stream)
    return _paged_attention(cache, batch, q, causal, scale, stream)


def _paged_attention(cache, batch, q, causal, scale, stream):
    if scale is None:
        scale = 1.0 / math.sqrt(cache.d)
    o = _torch.empty(q.shape, dtype=q.dtype, device=q.device)
    lse = _torch.empty(q.shape[:2], dtype=_F32, device=q.device)
    fa_forward_paged(cache, batch, q, o, lse, scale, causal, paged_workspace(cache, batch, q),
                     stream)
    return o, lse
