"""Score-modified attention: binding of ``calibatt_attn_spans``,
``calibatt_score_attn_fwd`` and ``calibatt_score_attn_bwd``.

Attention whose scores are capped by a tanh, biased by distance (a slope a
head, a learned table of buckets) and restricted to documents, a prefix or
lengths, on the kept blocks of a calibrated mask where one is given; with its
gradients, the table's included.  The definition stands in
``include/calibatt.h``.  As everywhere in this package the module checks and
marshals arguments, allocates outputs and workspace and passes the stream.
"""

from __future__ import annotations

import ctypes
import functools
import math
from dataclasses import dataclass

import numpy as np
import torch

from . import _lib
from ._lib import BF16, FP32, check, load

_DTYPES = {torch.bfloat16: BF16, torch.float32: FP32}


def _ptr(t):
    return None if t is None else t.data_ptr()


def _stream(device):
    # torch.cuda.current_stream builds a Stream object around this number (3 us a call)
    return torch._C._cuda_getCurrentRawStream(device.index)


def _on_device(device, call):
    """Runs ``call`` with ``device`` current (the usual case, that it is already, costs no context manager)."""
    if torch.cuda.current_device() == device.index:
        return call()
    with torch.cuda.device(device):
        return call()


@dataclass
class AttnSpans:
    """Visible keys of every query row (see ``calibatt_spans``), from :func:`attn_spans`."""

    B: int
    Nq: int
    Nk: int
    row: torch.Tensor       # [B, Nq, 2] int32: first visible key, one past the last
    tile: torch.Tensor      # [B, ceil(Nq / 128), 4] int32: ranges of 128-row tiles
    q_start: torch.Tensor   # [B] int32: key position of query row 0

    def as_struct(self):
        s = _lib.Spans()
        s.B, s.Nq, s.Nk = self.B, self.Nq, self.Nk
        s.row, s.tile, s.q_start = self.row.data_ptr(), self.tile.data_ptr(), self.q_start.data_ptr()
        return s


def _int32(x):
    """``x`` as the C interface's int: ctypes would wrap a wider one into range, clamped it is refused there."""
    return max(-(1 << 31), min(int(x), (1 << 31) - 1))


def _ints(name, x, shape, device):
    """int32 CUDA tensor of ``shape`` (None: not given); lists and host tensors are copied to the device."""
    if x is None:
        return None
    t = torch.as_tensor(x)
    if t.is_floating_point() or t.is_complex() or t.dtype == torch.bool:
        raise ValueError(f"{name} must hold integers")
    if tuple(t.shape) != shape:
        raise ValueError(f"{name} must have shape {shape}, got {tuple(t.shape)}")
    if t.is_cuda and t.device != device:
        raise ValueError(f"{name} must be on {device}")
    if t.dtype in (torch.int64, torch.uint32, torch.uint64):   # lengths are clamped on the device; a wrapped value would not be
        w = t.to(torch.int64)
        if t.dtype == torch.uint64:
            w = w.masked_fill(w < 0, 1 << 31)
        t = w.clamp(-(1 << 31), (1 << 31) - 1)
    return t.to(device=device, dtype=torch.int32).contiguous()


def attn_spans(B, Nq, Nk, *, causal=False, docs=None, prefix=None, kv_len=None, q_len=None, q_start=None,
               device="cuda"):
    """The keys every query row sees (``calibatt_attn_spans``), as one interval a row.

    Row i of batch entry b stands at key position ``q_start[b] + i`` (default
    0; a single new token: its position).  It sees the ``kv_len[b]`` keys of
    its batch entry, or with ``docs`` ([B, n_docs + 1] ascending bounds of
    documents packed back to back) those of its document; with ``causal`` only
    keys up to its own position and the first ``prefix[b, m]`` keys of its
    document ([B, n_docs], or [B] without documents).  Rows from ``q_len[b]``
    on see nothing.  Make it once per batch layout; every layer's calls share it.
    """
    B, Nq, Nk = int(B), int(Nq), int(Nk)
    if B <= 0 or Nq <= 0 or Nk <= 0:
        raise ValueError("B, Nq and Nk must be positive")
    if max(B, Nq, Nk) >= 1 << 31:
        raise ValueError("B, Nq and Nk must be below 2^31")
    device = torch.device(device)
    if device.type != "cuda":
        raise ValueError("the spans are computed on a CUDA device")
    if device.index is None:
        device = torch.device("cuda", torch.cuda.current_device())
    if prefix is not None and not causal:
        raise ValueError("a prefix needs causal=True")
    n_docs = 0
    if docs is not None:
        docs = torch.as_tensor(docs)
        if docs.dim() != 2 or docs.shape[0] != B or docs.shape[1] < 2:
            raise ValueError(f"docs must be [B, n_docs + 1] with B = {B}")
        n_docs = docs.shape[1] - 1
        docs = _ints("docs", docs, (B, n_docs + 1), device)
    if prefix is not None:
        prefix = torch.as_tensor(prefix)
        if n_docs == 0 and prefix.dim() == 1:
            prefix = prefix[:, None]
        prefix = _ints("prefix", prefix, (B, max(n_docs, 1)), device)
    kv_len = _ints("kv_len", kv_len, (B,), device)
    q_len = _ints("q_len", q_len, (B,), device)
    q_start = _ints("q_start", q_start, (B,), device)
    sp = AttnSpans(B, Nq, Nk, torch.empty((B, Nq, 2), dtype=torch.int32, device=device),
                   torch.empty((B, -(-Nq // 128), 4), dtype=torch.int32, device=device),
                   torch.empty(B, dtype=torch.int32, device=device))
    check(_on_device(device, lambda: load().calibatt_attn_spans(
        B, Nq, Nk, int(bool(causal)), _ptr(docs), n_docs, _ptr(prefix), _ptr(kv_len), _ptr(q_len), _ptr(q_start),
        _ptr(sp.row), _ptr(sp.tile), _ptr(sp.q_start), _stream(device))))
    return sp


def relative_buckets(n_buckets, max_distance, bidirectional=True, device="cuda"):
    """Bucket map [2 max_distance + 1] int32 of a learned relative bias (``calibatt_relative_buckets``):
    own buckets near zero, logarithmic ones out to ``max_distance``, farther offsets in the last."""
    n = int(max_distance) if 0 < int(max_distance) <= 1 << 20 else 0   # (others are refused before anything is written)
    out = np.zeros(2 * n + 1, dtype=np.int32)
    check(load().calibatt_relative_buckets(_int32(n_buckets), _int32(max_distance), int(bool(bidirectional)),
                                           out.ctypes.data_as(ctypes.c_void_p)))
    return torch.from_numpy(out).to(device)


def _tensor4(name, t, shape, dtype, device):
    """Checks a [B, heads, N, d] tensor and returns its ``calibatt_tensor4``."""
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {shape}, got {t.dtype} of shape {tuple(t.shape)}")
    if t.device != device or not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor on {device}")
    sb, sh, sn, sd = t.stride()
    step = 16 // t.element_size()
    if (sd != 1 or (shape[0] > 1 and (sb <= 0 or sb % step)) or (shape[1] > 1 and (sh <= 0 or sh % step))
            or (shape[2] > 1 and (sn <= 0 or sn % step))):
        raise ValueError(f"{name}: the last dimension must be contiguous and the others' strides positive multiples "
                         f"of 16 bytes, got strides {t.stride()} (an expanded tensor needs .contiguous())")
    return _lib.Tensor4(t.data_ptr(), sb, sh, sn)


def _flat(name, t, shape, dtype, device):
    """Checks a contiguous operand (None: not given)."""
    if t is None:
        return
    if t.shape != shape or t.dtype != dtype:
        raise ValueError(f"{name} must be {dtype} of shape {shape}, got {t.dtype} of shape {tuple(t.shape)}")
    if not t.is_cuda or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous CUDA tensor on {device}")


def _prepare(q, k, v, spans, scale, cap, slopes, table, buckets, mask, map_offset, status):
    """Argument checks shared by the forward and the backward: sizes, the score struct and its operands."""
    if q.dim() != 4 or k.dim() != 4:
        raise ValueError("q must be [B, H, Nq, d] and k, v [B, Hkv, Nk, d]")
    if q.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {q.dtype}: use torch.bfloat16 or torch.float32")
    B, H, Nq, d = q.shape
    Hkv, Nk = k.shape[1], k.shape[2]
    if Hkv == 0 or H % Hkv:
        raise ValueError(f"H = {H} must be a multiple of Hkv = {Hkv}")
    if not isinstance(spans, AttnSpans):
        raise TypeError("spans must come from attn_spans")
    if (spans.B, spans.Nq, spans.Nk) != (B, Nq, Nk):
        raise ValueError(f"spans of B, Nq, Nk = {spans.B, spans.Nq, spans.Nk} do not match {B, Nq, Nk}")
    dev = q.device
    _flat("spans.row", spans.row, (B, Nq, 2), torch.int32, dev)
    _flat("spans.tile", spans.tile, (B, -(-Nq // 128), 4), torch.int32, dev)
    _flat("spans.q_start", spans.q_start, (B,), torch.int32, dev)
    if (table is None) != (buckets is None):
        raise ValueError("table and buckets come together")
    sc = _lib.Score()
    sc.scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    sc.cap = float(cap)
    _flat("slopes", slopes, (H,), torch.float32, dev)
    sc.slopes = None if slopes is None else slopes.data_ptr()
    if table is not None:
        if table.dim() != 2 or buckets.dim() != 1 or buckets.numel() % 2 == 0:
            raise ValueError("table must be [H, n_buckets] and buckets [2 max_distance + 1]")
        _flat("table", table, (H, table.shape[1]), q.dtype, dev)
        _flat("buckets", buckets, tuple(buckets.shape), torch.int32, dev)
        sc.table, sc.buckets = table.data_ptr(), buckets.data_ptr()
        sc.n_buckets, sc.max_distance = _int32(table.shape[1]), _int32(buckets.numel() // 2)
    if mask is not None:
        if mask.dim() != 3:
            raise ValueError("mask must be uint8 [n_maps, nqb, nkb]")
        _flat("mask", mask, (mask.shape[0], -(-Nq // 128), -(-Nk // 128)), torch.uint8, dev)
        sc.mask, sc.n_maps, sc.map_offset = mask.data_ptr(), mask.shape[0], _int32(map_offset)
    if status is not None:
        if status.dtype != torch.int32 or status.numel() < 1:
            raise ValueError("status must be an int32 tensor with at least one element")
        _flat("status", status, tuple(status.shape), torch.int32, dev)
    return (B, H, Hkv, Nq, Nk, d), sc


@functools.lru_cache(maxsize=1024)
def _fwd_bytes(*sizes):
    n = ctypes.c_size_t(0)
    check(load().calibatt_score_attn_fwd_workspace_size(*sizes, ctypes.byref(n)))
    return n.value


@functools.lru_cache(maxsize=1024)
def _bwd_bytes(*sizes):
    n = ctypes.c_size_t(0)
    check(load().calibatt_score_attn_bwd_workspace_size(*sizes, ctypes.byref(n)))
    return n.value


def _workspace(nbytes, device):
    return torch.empty(nbytes, dtype=torch.uint8, device=device) if nbytes else None


def score_attn_fwd(q, k, v, spans: AttnSpans, *, scale=None, cap=0.0, slopes=None, table=None, buckets=None, mask=None,
                   map_offset=0, return_lse=False, out=None, lse=None, status=None):
    """Score-modified attention forward (``calibatt_score_attn_fwd``).

    q: [B, H, Nq, d]; k, v: [B, Hkv, Nk, d], bf16 or fp32 on the GPU, H a
    multiple of Hkv, d 64 or 128, any strides with the last dimension
    contiguous and 16-byte aligned rows.  ``spans``: the keys every row sees
    (:func:`attn_spans`).  Scores: scale q.k (scale 1/sqrt(d) when None),
    capped to cap tanh(s / cap) when ``cap`` > 0, minus ``slopes``[h] |j - p|
    ([H] float32; rows that see keys farther away than 2^24 become NaN and are
    reported to ``status``), plus ``table``[h, buckets[j - p]] ([H, n_buckets] of q's
    type; ``buckets`` int32 [2 max_distance + 1], e.g. from
    :func:`relative_buckets`).  ``mask``: uint8 [n_maps, nqb, nkb] kept 128 x
    128 blocks (as :func:`calibrate` returns), head h uses map ``map_offset``
    + h.  Returns O (laid out like q) and, with ``return_lse``, LSE [B, H, Nq].

    With gradients enabled and an input that requires one, O is part of the
    graph: its backward is :func:`score_attn_bwd`, for q, k, v and the table.
    (With ``out`` the returned tensor is, ``out`` itself stays outside.)  The
    LSE and the slopes have no gradient; a backward that asks for one raises.
    """
    if torch.is_grad_enabled() and (q.requires_grad or k.requires_grad or v.requires_grad
                                    or (table is not None and table.requires_grad)
                                    or (slopes is not None and slopes.requires_grad)):
        o, lse = _ScoreAttention.apply(q, k, v, table, slopes, spans, out, lse,
                                       dict(scale=scale, cap=cap, buckets=buckets, mask=mask, map_offset=map_offset,
                                            status=status))
        return (o, lse) if return_lse else o
    (B, H, Hkv, Nq, Nk, d), sc = _prepare(q, k, v, spans, scale, cap, slopes, table, buckets, mask, map_offset, status)
    dev, dt = q.device, q.dtype
    tq = _tensor4("q", q, (B, H, Nq, d), dt, dev)
    tk = _tensor4("k", k, (B, Hkv, Nk, d), dt, dev)
    tv = _tensor4("v", v, (B, Hkv, Nk, d), dt, dev)
    if out is None:
        out = torch.empty_like(q)
    to = _tensor4("out", out, (B, H, Nq, d), dt, dev)
    if return_lse and lse is None:
        lse = torch.empty((B, H, Nq), device=dev, dtype=torch.float32)
    _flat("lse", lse, (B, H, Nq), torch.float32, dev)
    sizes = (B, H, Hkv, Nq, Nk, d, _DTYPES[dt])
    nbytes = _fwd_bytes(*sizes)
    ws = _workspace(nbytes, dev)
    ref = ctypes.byref
    sp = spans.as_struct()
    check(_on_device(dev, lambda: load().calibatt_score_attn_fwd(
        ref(tq), ref(tk), ref(tv), ref(to), _ptr(lse), *sizes, ref(sp), ref(sc), _ptr(ws), nbytes, _ptr(status),
        _stream(dev))))
    return (out, lse) if return_lse else out


def score_attn_bwd(dout, q, k, v, o, lse, spans: AttnSpans, *, scale=None, cap=0.0, slopes=None, table=None,
                   buckets=None, mask=None, map_offset=0, status=None):
    """Gradients of :func:`score_attn_fwd` (``calibatt_score_attn_bwd``).

    ``dout``: gradient of O; ``o``, ``lse``: the forward's results; the other
    arguments as given to the forward.  Returns (dq, dk, dv), laid out like q,
    k and v, and the table's gradient [H, n_buckets] as fourth where a table
    is given.  Deterministic.
    """
    (B, H, Hkv, Nq, Nk, d), sc = _prepare(q, k, v, spans, scale, cap, slopes, table, buckets, mask, map_offset, status)
    dev, dt = q.device, q.dtype
    qs, ks = (B, H, Nq, d), (B, Hkv, Nk, d)
    ins = [_tensor4("dout", dout, qs, dt, dev), _tensor4("q", q, qs, dt, dev), _tensor4("k", k, ks, dt, dev),
           _tensor4("v", v, ks, dt, dev), _tensor4("o", o, qs, dt, dev)]
    _flat("lse", lse, (B, H, Nq), torch.float32, dev)
    if lse is None:
        raise ValueError("lse must be the forward's (return_lse=True)")
    dq, dk, dv = torch.empty_like(q), torch.empty_like(k), torch.empty_like(v)
    outs = [_tensor4("dq", dq, qs, dt, dev), _tensor4("dk", dk, ks, dt, dev), _tensor4("dv", dv, ks, dt, dev)]
    dtable = None if table is None else torch.empty_like(table)
    sizes = (B, H, Hkv, Nq, Nk, d, _DTYPES[dt])
    nbytes = _bwd_bytes(*sizes, 0 if table is None else _int32(table.shape[1]))
    ws = _workspace(nbytes, dev)
    ref = ctypes.byref
    sp = spans.as_struct()
    check(_on_device(dev, lambda: load().calibatt_score_attn_bwd(
        *map(ref, ins), _ptr(lse), *map(ref, outs), _ptr(dtable), *sizes, ref(sp), ref(sc), _ptr(ws), nbytes,
        _ptr(status), _stream(dev))))
    return (dq, dk, dv) if table is None else (dq, dk, dv, dtable)


class _ScoreAttention(torch.autograd.Function):
    """:func:`score_attn_fwd` as a node of the graph."""

    @staticmethod
    def forward(ctx, q, k, v, table, slopes, spans, out, lse, kw):
        # The caller's buffers enter as aliases: marked as written, so that an
        # older graph that saved them notices, but without a history of their
        # own, which would chain the graphs of calls that share them.
        given = [t for t in (out, lse) if t is not None]
        out, lse = (None if t is None else t.detach() for t in (out, lse))
        o, lse = score_attn_fwd(q, k, v, spans, table=table, slopes=slopes, out=out, lse=lse, return_lse=True, **kw)
        torch.autograd.graph.increment_version(given)
        ctx.save_for_backward(q, k, v, table, slopes, o, lse)
        ctx.spans, ctx.kw = spans, kw
        ctx.set_materialize_grads(False)
        return o, lse

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dout, dlse):
        if dlse is not None:
            raise RuntimeError("the LSE of score_attn_fwd has no gradient: use it detached")
        if ctx.needs_input_grad[4]:
            raise RuntimeError("the slopes of score_attn_fwd have no gradient: pass them detached")
        if dout is None:
            return (None,) * 9
        q, k, v, table, slopes, o, lse = ctx.saved_tensors
        try:
            _tensor4("dout", dout, q.shape, q.dtype, q.device)
        except ValueError:   # strides that the kernels do not take (a sum's gradient is expanded)
            dout = dout.contiguous()
        if dout.data_ptr() % 16:
            dout = dout.clone()
        grads = score_attn_bwd(dout, q, k, v, o, lse, ctx.spans, table=table, slopes=slopes, **ctx.kw)
        dq, dk, dv = (g if need else None for g, need in zip(grads[:3], ctx.needs_input_grad))
        return dq, dk, dv, grads[3] if ctx.needs_input_grad[3] else None, None, None, None, None, None
