"""Binding of include/rd_moe.h: the operators around the grouped expert products.

Argument marshalling only, as in the package itself (whose functions these are, too):

* ``route(logits, topk, ...)``                        -> Routing(ids, weights, group_sizes, pos, rows)
* ``route_bwd(logits, ids, d_weights, ...)``          -> d_logits
* ``sort_rows(ids, experts, ...)``                    -> (group_sizes, pos, rows)
* ``dispatch_rows(x, pos, ...)``                      -> packed rows; its gradient is combine_rows
* ``combine_rows(y, pos, w, ...)``                    -> token rows
* ``combine_rows_bwd(d_out, y, pos, w, ...)``         -> (d_y, d_w)
* ``mxfp4_quantize(x, pos=None, ...)``                -> Mxfp4(q, scales), 4-bit microscaled rows
* ``mxfp4_quantize_weights(rhs, ...)``                -> Mxfp4 of expert weights [g, k, n]
* ``mxfp4_dequantize(q, scales, ...)``                -> bf16 rows
* ``ragged_dot_mxfp4(a, a_scales, b, b_scales, group_sizes, ...)`` -> the grouped product

A layer: ``route`` the tokens, ``dispatch_rows`` (or ``mxfp4_quantize(x, pos=...)``) them into the
packed buffer, run the grouped products with ``group_sizes``, ``combine_rows`` the result.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import expert_ffn_ragged_gb300 as _rd

SCORE_SOFTMAX = 0
SCORE_SIGMOID = 1
MAX_TOPK = 32
MAX_EXPERT_GROUPS = 32
EPI_SILU_GLU_MXFP4 = 2

_F32, _BF16 = 0, 1


class Routing(NamedTuple):
    """What ``route`` gives: ids / weights / pos [tokens, topk], group_sizes [experts], rows [1]."""

    ids: object
    weights: object
    group_sizes: object
    pos: object
    rows: object


class Mxfp4(NamedTuple):
    """4-bit rows: q [..., k / 2] and scales [..., mxfp4_scale_width(k)], both uint8."""

    q: object
    scales: object


class _RouteConfig(ctypes.Structure):
    _fields_ = [("topk", ctypes.c_int32), ("score", ctypes.c_int32), ("groups", ctypes.c_int32),
                ("topk_groups", ctypes.c_int32), ("renormalize", ctypes.c_int32),
                ("scale", ctypes.c_float)]


def declare(lib):
    """Argument and result types of the entry points of rd_moe.h."""
    vp, i64, i32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32
    for name, args in (
            ("rd_route", [vp, i32, vp, i64, i64, vp, vp, vp, vp, vp, vp, vp, vp]),
            ("rd_route_bwd", [vp, i32, vp, vp, i64, i64, vp, vp, vp, vp]),
            ("rd_sort_rows", [vp, i64, i64, i64, vp, vp, vp, vp, vp]),
            ("rd_dispatch_rows", [vp, vp, vp, i64, i64, i64, i64, vp, vp]),
            ("rd_combine_rows", [vp, vp, vp, vp, i64, i64, i64, i64, vp, vp]),
            ("rd_combine_rows_bwd", [vp, vp, vp, vp, vp, vp, i64, i64, i64, i64, vp, vp]),
            ("rd_mxfp4_quantize", [vp, vp, vp, vp, i64, i64, i64, i64, vp, vp]),
            ("rd_mxfp4_quantize_weights", [vp, vp, vp, i64, i64, i64, vp]),
            ("rd_mxfp4_dequantize", [vp, vp, vp, i64, i64, vp, vp]),
            ("rd_ragged_dot_mxfp4", [vp] * 6 + [i64, i64, i64, vp, i32, i32, i32, vp, i32, vp, vp])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


def _check_tensor(t, name, shape, dtype):
    """t must be a contiguous CUDA tensor of this dtype and shape (None: any extent)."""
    if (t.dtype != dtype or t.dim() != len(shape) or not t.is_cuda or not t.is_contiguous()
            or any(w is not None and w != g for w, g in zip(shape, t.shape))):
        raise ValueError(f"{name} must be a contiguous {dtype} CUDA tensor of shape "
                         f"{['any' if w is None else w for w in shape]}")


def _given(t, name, shape, dtype, device):
    """The caller's output buffer after its checks, or a new one."""
    if t is None:
        return _rd._torch().empty(shape, dtype=dtype, device=device)
    _check_tensor(t, name, shape, dtype)
    return t


def _logits_type(logits):
    torch = _rd._torch()
    if logits.dtype not in (torch.float32, torch.bfloat16):
        raise ValueError("logits must be float32 or bfloat16")
    _check_tensor(logits, "logits", (None, None), logits.dtype)
    return _F32 if logits.dtype == torch.float32 else _BF16


def route(logits, topk: int, score: int = SCORE_SOFTMAX, bias=None, groups: int = 1,
          topk_groups: Optional[int] = None, renormalize: bool = True, scale: float = 1.0, limit=None,
          out: Optional[Routing] = None, stream=None) -> Routing:
    """Router logits [tokens, experts] to expert ids, weights and the packed buffer's plan (rd_route).

    ``topk_groups`` defaults to all groups.  ``out``: a Routing of buffers to write into.
    """
    torch = _rd._torch()
    lib = _rd.load()
    dtype = _logits_type(logits)
    tokens, experts = logits.shape
    dev = logits.device
    if bias is not None:
        _check_tensor(bias, "bias", (experts,), torch.float32)
    _rd._scalar_i32(limit, "limit")
    o = out if out is not None else Routing(None, None, None, None, None)
    i32 = torch.int32
    r = Routing(_given(o.ids, "ids", (tokens, topk), i32, dev),
                _given(o.weights, "weights", (tokens, topk), torch.float32, dev),
                _given(o.group_sizes, "group_sizes", (experts,), i32, dev),
                _given(o.pos, "pos", (tokens, topk), i32, dev),
                _given(o.rows, "rows", (1,), i32, dev))
    _rd._same_device(dev, bias, limit, *r)
    cfg = _RouteConfig(int(topk), int(score), int(groups),
                       int(groups if topk_groups is None else topk_groups), int(bool(renormalize)),
                       float(scale))
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_route(ptr(logits), dtype, ptr(bias), tokens, experts, ctypes.byref(cfg),
                            ptr(limit), ptr(r.ids), ptr(r.weights), ptr(r.group_sizes), ptr(r.pos),
                            ptr(r.rows), _rd._stream(stream, dev))
    _rd._check(code, "rd_route")
    return r


def route_bwd(logits, ids, d_weights, score: int = SCORE_SOFTMAX, renormalize: bool = True,
              scale: float = 1.0, limit=None, out=None, stream=None):
    """Gradient of the logits from that of the weights (rd_route_bwd); settings as in ``route``."""
    torch = _rd._torch()
    lib = _rd.load()
    dtype = _logits_type(logits)
    tokens, experts = logits.shape
    dev = logits.device
    _check_tensor(ids, "ids", (tokens, None), torch.int32)
    _check_tensor(d_weights, "d_weights", tuple(ids.shape), torch.float32)
    _rd._scalar_i32(limit, "limit")
    out = _given(out, "out", (tokens, experts), logits.dtype, dev)
    _rd._same_device(dev, ids, d_weights, limit, out)
    cfg = _RouteConfig(ids.shape[1], int(score), 1, 1, int(bool(renormalize)), float(scale))
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_route_bwd(ptr(logits), dtype, ptr(ids), ptr(d_weights), tokens, experts,
                                ctypes.byref(cfg), ptr(limit), ptr(out), _rd._stream(stream, dev))
    _rd._check(code, "rd_route_bwd")
    return out


def sort_rows(ids, experts: int, limit=None, stream=None):
    """(group_sizes [experts], pos [tokens, topk], rows [1]) of expert ids (rd_sort_rows)."""
    torch = _rd._torch()
    lib = _rd.load()
    _check_tensor(ids, "ids", (None, None), torch.int32)
    _rd._scalar_i32(limit, "limit")
    tokens, topk = ids.shape
    dev = ids.device
    sizes = torch.empty((max(int(experts), 0),), dtype=torch.int32, device=dev)
    pos = torch.empty_like(ids)
    rows = torch.empty((1,), dtype=torch.int32, device=dev)
    _rd._same_device(dev, limit)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_sort_rows(ptr(ids), tokens, topk, int(experts), ptr(limit), ptr(sizes), ptr(pos),
                                ptr(rows), _rd._stream(stream, dev))
    _rd._check(code, "rd_sort_rows")
    return sizes, pos, rows


def dispatch_rows(x, pos, out_rows: Optional[int] = None, limit=None, out=None, stream=None):
    """out[pos[t, k]] = x[t] (rd_dispatch_rows); out_rows defaults to tokens * topk."""
    torch = _rd._torch()
    lib = _rd.load()
    _check_tensor(x, "x", (None, None), torch.bfloat16)
    tokens, hidden = x.shape
    _check_tensor(pos, "pos", (tokens, None), torch.int32)
    _rd._scalar_i32(limit, "limit")
    topk, dev = pos.shape[1], x.device
    n = tokens * topk if out_rows is None else int(out_rows)
    if out is not None and out_rows is None:
        n = out.shape[0]
    out = _given(out, "out", (n, hidden), torch.bfloat16, dev)
    _rd._same_device(dev, pos, limit, out)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_dispatch_rows(ptr(x), ptr(pos), ptr(out), tokens, topk, hidden, n, ptr(limit),
                                    _rd._stream(stream, dev))
    _rd._check(code, "rd_dispatch_rows")
    return out


def combine_rows(y, pos, w=None, limit=None, out=None, stream=None):
    """out[t] = sum_k w[t, k] y[pos[t, k]] (rd_combine_rows); without ``w`` every weight is one."""
    torch = _rd._torch()
    lib = _rd.load()
    _check_tensor(y, "y", (None, None), torch.bfloat16)
    _check_tensor(pos, "pos", (None, None), torch.int32)
    tokens, topk = pos.shape
    if w is not None:
        _check_tensor(w, "w", (tokens, topk), torch.float32)
    _rd._scalar_i32(limit, "limit")
    rows, hidden = y.shape
    dev = y.device
    out = _given(out, "out", (tokens, hidden), torch.bfloat16, dev)
    _rd._same_device(dev, pos, w, limit, out)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_combine_rows(ptr(y), ptr(pos), ptr(w), ptr(out), tokens, topk, hidden, rows,
                                   ptr(limit), _rd._stream(stream, dev))
    _rd._check(code, "rd_combine_rows")
    return out


def combine_rows_bwd(d_out, y, pos, w, limit=None, d_y=None, d_w=None, stream=None):
    """(d_y, d_w) of ``combine_rows`` (rd_combine_rows_bwd)."""
    torch = _rd._torch()
    lib = _rd.load()
    _check_tensor(y, "y", (None, None), torch.bfloat16)
    rows, hidden = y.shape
    _check_tensor(d_out, "d_out", (None, hidden), torch.bfloat16)
    tokens = d_out.shape[0]
    _check_tensor(pos, "pos", (tokens, None), torch.int32)
    topk = pos.shape[1]
    _check_tensor(w, "w", (tokens, topk), torch.float32)
    _rd._scalar_i32(limit, "limit")
    dev = y.device
    d_y = _given(d_y, "d_y", (rows, hidden), torch.bfloat16, dev)
    d_w = _given(d_w, "d_w", (tokens, topk), torch.float32, dev)
    _rd._same_device(dev, d_out, pos, w, limit, d_y, d_w)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_combine_rows_bwd(ptr(d_out), ptr(y), ptr(pos), ptr(w), ptr(d_y), ptr(d_w), tokens,
                                       topk, hidden, rows, ptr(limit), _rd._stream(stream, dev))
    _rd._check(code, "rd_combine_rows_bwd")
    return d_y, d_w


def mxfp4_scale_width(k: int) -> int:
    """Bytes of one row's scales: k / 32 rounded up to a multiple of 16 (rd_mxfp4_scale_width)."""
    return 0 if k <= 0 else (k // 32 + 15) // 16 * 16


def mxfp4_quantize(x, pos=None, out_rows: Optional[int] = None, limit=None,
                   out: Optional[Mxfp4] = None, stream=None) -> Mxfp4:
    """bf16 rows [rows, k] to 4-bit rows; with ``pos`` straight to their packed rows (rd_mxfp4_quantize)."""
    torch = _rd._torch()
    lib = _rd.load()
    _check_tensor(x, "x", (None, None), torch.bfloat16)
    rows, k = x.shape
    dev = x.device
    topk = 1
    if pos is not None:
        _check_tensor(pos, "pos", (rows, None), torch.int32)
        topk = pos.shape[1]
    _rd._scalar_i32(limit, "limit")
    n = rows * topk if out_rows is None else int(out_rows)
    o = out if out is not None else Mxfp4(None, None)
    if out is not None and out_rows is None:
        n = out.q.shape[0]
    q = _given(o.q, "q", (n, k // 2), torch.uint8, dev)
    scales = _given(o.scales, "scales", (n, mxfp4_scale_width(k)), torch.uint8, dev)
    _rd._same_device(dev, pos, limit, q, scales)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_mxfp4_quantize(ptr(x), ptr(pos), ptr(q), ptr(scales), rows, topk, k, n, ptr(limit),
                                     _rd._stream(stream, dev))
    _rd._check(code, "rd_mxfp4_quantize")
    return Mxfp4(q, scales)


def mxfp4_quantize_weights(rhs, out: Optional[Mxfp4] = None, stream=None) -> Mxfp4:
    """Expert weights [g, k, n] bf16 to 4-bit rows along k: q [g, n, k / 2] (rd_mxfp4_quantize_weights)."""
    torch = _rd._torch()
    lib = _rd.load()
    _check_tensor(rhs, "rhs", (None, None, None), torch.bfloat16)
    g, k, n = rhs.shape
    dev = rhs.device
    o = out if out is not None else Mxfp4(None, None)
    q = _given(o.q, "q", (g, n, k // 2), torch.uint8, dev)
    scales = _given(o.scales, "scales", (g, n, mxfp4_scale_width(k)), torch.uint8, dev)
    _rd._same_device(dev, q, scales)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_mxfp4_quantize_weights(ptr(rhs), ptr(q), ptr(scales), g, k, n,
                                             _rd._stream(stream, dev))
    _rd._check(code, "rd_mxfp4_quantize_weights")
    return Mxfp4(q, scales)


def mxfp4_dequantize(q, scales, limit=None, out=None, stream=None):
    """The values of 4-bit rows [rows, k / 2] as bf16 [rows, k] (rd_mxfp4_dequantize)."""
    torch = _rd._torch()
    lib = _rd.load()
    _check_tensor(q, "q", (None, None), torch.uint8)
    rows, k = q.shape[0], 2 * q.shape[1]
    _check_tensor(scales, "scales", (rows, mxfp4_scale_width(k)), torch.uint8)
    _rd._scalar_i32(limit, "limit")
    dev = q.device
    out = _given(out, "out", (rows, k), torch.bfloat16, dev)
    _rd._same_device(dev, scales, limit, out)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_mxfp4_dequantize(ptr(q), ptr(scales), ptr(out), rows, k, ptr(limit),
                                       _rd._stream(stream, dev))
    _rd._check(code, "rd_mxfp4_dequantize")
    return out


def ragged_dot_mxfp4(a, a_scales, b, b_scales, group_sizes, group_offset: int = 0, limit=None,
                     epilogue: int = 0, out=None, out_scales=None, status=None, stream=None):
    """Grouped product of 4-bit rows a [m, k / 2] and weights b [g_local, n, k / 2] (rd_ragged_dot_mxfp4).

    EPI_NONE and EPI_SILU_GLU give bf16 rows, EPI_SILU_GLU_MXFP4 an Mxfp4 of 4-bit rows.
    """
    torch = _rd._torch()
    lib = _rd.load()
    u8 = torch.uint8
    _check_tensor(a, "a", (None, None), u8)
    m, k = a.shape[0], 2 * a.shape[1]
    _check_tensor(b, "b", (None, None, k // 2), u8)
    g_local, n = b.shape[0], b.shape[1]
    width = mxfp4_scale_width(k)
    _check_tensor(a_scales, "a_scales", (m, width), u8)
    _check_tensor(b_scales, "b_scales", (g_local, n, width), u8)
    _rd._group_args(group_sizes, limit, status)
    dev = a.device
    if epilogue == EPI_SILU_GLU_MXFP4:
        out = _given(out, "out", (m, n // 4), u8, dev)
        out_scales = _given(out_scales, "out_scales", (m, mxfp4_scale_width(n // 2)), u8, dev)
    else:
        if out_scales is not None:
            raise ValueError("out_scales belongs to EPI_SILU_GLU_MXFP4")
        out = _given(out, "out", (m, n // 2 if epilogue == _rd.EPI_SILU_GLU else n), torch.bfloat16, dev)
    _rd._same_device(dev, a_scales, b, b_scales, group_sizes, limit, status, out, out_scales)
    ptr = _rd._ptr
    with _rd._on_device(dev):
        code = lib.rd_ragged_dot_mxfp4(ptr(a), ptr(a_scales), ptr(b), ptr(b_scales), ptr(out),
                                       ptr(out_scales), m, k, n, ptr(group_sizes), group_sizes.numel(),
                                       int(group_offset), g_local, ptr(limit), int(epilogue),
                                       ptr(status), _rd._stream(stream, dev))
    _rd._check(code, "rd_ragged_dot_mxfp4")
    return out if out_scales is None else Mxfp4(out, out_scales)
