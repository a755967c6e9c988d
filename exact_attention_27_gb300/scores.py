"""Binding of the shaped-score entry points of include/fa.h.

`Scores` says what is done to a score (of a model or a layer), `KeySpans` which keys each query
sees (of a step's batch).  Like the other handles they hold tensors, not values: spans written in
place are seen by the next call, and a captured graph replays with what the tensors then hold.

fa_forward_scores and fa_backward_scores write into the caller's tensors; attention_forward and
attention_backward take `scores` and `spans` and allocate what they return.
"""

import ctypes
import math

from . import _lib, paged
from ._lib import FaError, int32, library
from .paged import _byref, _load_torch, _same_device, _stream


class Scores:
    """What is done to a score scale q.k: softcap tanh(x / softcap) (0: nothing), then less
    slopes[h] times the distance of the two positions (slopes [H_q] fp32 on the GPU, None:
    nothing; they get no gradient), and `window`, the last positions that a query sees, its own
    among them (0: all)."""

    def __init__(self, softcap=0.0, slopes=None, window=0):
        torch = _load_torch()
        softcap, window = float(softcap), int(window)
        held = ctypes.c_float(softcap).value  # (0 means no cap, so that none may round to it)
        if not math.isfinite(held) or softcap < 0 or (held == 0) != (softcap == 0):
            raise ValueError(f"softcap {softcap}: finite and >= 0 in fp32 is needed")
        if not 0 <= window < 2**31:
            raise ValueError(f"window {window}: 0 to 2**31 - 1 is needed")
        self.slopes, self.softcap, self.window, self.device = slopes, softcap, window, None
        if slopes is not None:
            if slopes.dtype is not torch.float32 or not slopes.is_cuda or slopes.dim() != 1 or \
                    not slopes.is_contiguous():
                raise ValueError("slopes must be a contiguous fp32 CUDA vector")
            self.device = slopes.get_device()
        self._c = _lib.ScoreSpec(softcap, slopes.data_ptr() if slopes is not None else None, window)
        self._ref = _byref(self._c)

    def _check(self, Hq, device):
        if self.slopes is not None:
            if self.slopes.shape[0] != Hq:
                raise ValueError(f"slopes has {self.slopes.shape[0]} values, expected {Hq}")
            if self.device != device:
                raise ValueError(f"slopes is on cuda:{self.device}, not cuda:{device}")


class KeySpans:
    """The keys that each query sees: first[b, i] <= j < end[b, i], int32 CUDA tensors [B, N_q], or
    [N_q] for all entries of a batch alike; None: from the first key, to the last.  The causal mask
    and the window of a call apply as well; rows that then see nothing get zeros."""

    def __init__(self, first=None, end=None):
        torch = _load_torch()
        given = [("first", first), ("end", end)]
        given = [(n, t) for n, t in given if t is not None]
        if not given:
            raise ValueError("give first, end or both")
        shapes, strides, devices = set(), set(), set()
        for name, t in given:
            if not isinstance(t, torch.Tensor) or t.dtype is not torch.int32 or not t.is_cuda or \
                    t.dim() not in (1, 2):
                raise ValueError(f"{name} must be an int32 CUDA tensor [B, N_q] or [N_q]")
            if t.shape[-1] > 1 and t.stride(-1) != 1:
                raise ValueError(f"{name} must be contiguous along its last dimension")
            shapes.add(tuple(t.shape))
            strides.add(t.stride(0) if t.dim() == 2 and t.shape[0] > 1 else 0)
            devices.add(t.get_device())
        if len(shapes) > 1 or len(strides) > 1 or len(devices) > 1:
            raise ValueError("first and end must have one shape, one stride and one device")
        self.first, self.end = first, end
        shape = shapes.pop()
        self.B, self.N = (1, shape[0]) if len(shape) == 1 else shape
        self.device = devices.pop()
        self._c = _lib.KeySpansStruct(*(t.data_ptr() if t is not None else None
                                        for t in (first, end)), strides.pop())
        self._ref = _byref(self._c)

    @classmethod
    def documents(cls, bounds, N_q):
        """Packed documents: bounds int32 [B, n + 1] or [n + 1], not decreasing; rows bounds[d] to
        bounds[d + 1] - 1 see the keys of the same places, rows outside all of them nothing."""
        torch = _load_torch()
        row = torch.arange(N_q, dtype=torch.int32, device=bounds.device)
        if bounds.dim() == 2:
            row = row.expand(bounds.shape[0], N_q).contiguous()
        d = torch.searchsorted(bounds.contiguous(), row, right=True, out_int32=True)
        n = bounds.shape[-1]
        inside = (d > 0) & (d < n)
        first = torch.gather(bounds, -1, (d - 1).clamp(0, n - 1).long())
        end = torch.gather(bounds, -1, d.clamp(0, n - 1).long())
        zero = torch.zeros_like(first)
        return cls(torch.where(inside, first, zero), torch.where(inside, end, zero))

    @classmethod
    def prefix(cls, lengths, N_q, q_offset=0):
        """A beginning that every query sees, of `lengths` [B] int32 keys, and the causal mask past
        it (the call itself is then not causal)."""
        torch = _load_torch()
        pos = torch.arange(q_offset + 1, q_offset + 1 + N_q, dtype=torch.int32,
                           device=lengths.device)
        return cls(None, torch.maximum(pos, lengths.to(torch.int32)[:, None]))

    @classmethod
    def lengths(cls, lengths, N_q):
        """A padded batch: the keys below lengths [B] int32."""
        torch = _load_torch()
        return cls(None, lengths.to(torch.int32)[:, None].expand(lengths.shape[0], N_q).contiguous())

    def _check(self, B, Nq, device):
        if self.N != Nq or self.B not in (1, B):
            raise ValueError(f"spans are [{self.B}, {self.N}], expected [{B}, {Nq}]")
        if self.device != device:
            raise ValueError(f"spans are on cuda:{self.device}, not cuda:{device}")


def _checked(q, k, named, lse, scores, spans):
    """Sizes of a call, after the checks that its tensors share."""
    torch = _load_torch()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, N, d]")
    B, Hq, Nq, d = q.shape
    if k.shape[0] != B or k.shape[3] != d:
        raise ValueError("k must be [B, H_kv, N_kv, d] with q's B and d")
    device = q.get_device()
    for name, t, like in [("q", q, q), ("k", k, k)] + named:
        if t.dtype is not torch.bfloat16 or not t.is_cuda or not t.is_contiguous():
            raise ValueError(f"{name} must be a contiguous bf16 CUDA tensor")
        if t.shape != like.shape:
            raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(like.shape)}")
        if t.get_device() != device:
            raise ValueError(f"{name} is on cuda:{t.get_device()}, not cuda:{device}")
    if lse.dtype is not torch.float32 or lse.get_device() != device or not lse.is_contiguous() or \
            lse.shape != (B, Hq, Nq):
        raise ValueError(f"lse must be a contiguous fp32 CUDA tensor {(B, Hq, Nq)}")
    if device != paged._device():
        _same_device(device)
    if scores is not None:
        scores._check(Hq, device)
    if spans is not None:
        spans._check(B, Nq, device)
    return device, B, Hq, k.shape[1], Nq, k.shape[2], d


def fa_forward_scores(q, k, v, o, lse, scale, causal, q_offset=0, scores=None, spans=None,
                      stream=None):
    """fa_forward_scores of include/fa.h: q [B, H_q, N_q, d] against k and v [B, H_kv, N_kv, d];
    writes o and lse."""
    q_offset = int32("q_offset", q_offset)
    device, *sizes = _checked(q, k, [("v", v, k), ("o", o, q)], lse, scores, spans)
    status = library().fa_forward_scores(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), *sizes,
        ctypes.c_float(scale), int(bool(causal)), q_offset,
        scores._ref if scores is not None else None, spans._ref if spans is not None else None,
        _stream(stream, device))
    if status:
        raise FaError(status, "fa_forward_scores")


def scores_workspace(q, k, causal, q_offset=0):
    """A workspace for fa_backward_scores calls of these sizes.  Its contents do not matter, and
    calls on one stream may share it; calls that can overlap, such as two captured graphs, may
    not."""
    torch = _load_torch()
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q and k must be [B, H, N, d]")
    B, Hq, Nq, d = q.shape
    n = library().fa_backward_scores_workspace_bytes(B, Hq, k.shape[1], Nq, k.shape[2], d,
                                                     int(bool(causal)),
                                                     int32("q_offset", q_offset))
    return torch.empty(n, dtype=torch.uint8, device=q.device)


def fa_backward_scores(q, k, v, o, lse, do, dq, dk, dv, scale, causal, workspace, q_offset=0,
                       scores=None, spans=None, stream=None):
    """fa_backward_scores of include/fa.h with the arguments of the forward that gave o and lse;
    writes dq, dk and dv."""
    q_offset = int32("q_offset", q_offset)
    device, *sizes = _checked(q, k, [("v", v, k), ("o", o, q), ("do", do, q), ("dq", dq, q),
                                     ("dk", dk, k), ("dv", dv, k)], lse, scores, spans)
    if workspace.get_device() != device or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on cuda:{device}")
    status = library().fa_backward_scores(
        q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), lse.data_ptr(), do.data_ptr(),
        dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), *sizes, ctypes.c_float(scale),
        int(bool(causal)), q_offset, scores._ref if scores is not None else None,
        spans._ref if spans is not None else None, workspace.data_ptr(), workspace.nbytes,
        _stream(stream, device))
    if status:
        raise FaError(status, "fa_backward_scores")
