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


# A call's host work is part of its latency, so the checks below are written out where a helper
# would cost more than it checks: dtype objects are compared by identity, shapes as tuples, devices
# as indices, and the settings of a router are marshalled once.  An argument's name stays bound to its
# tensor until the launch: it may be the last reference, and a new output would take its memory.

def _refuse(name, shape, dtype, idx):
    raise ValueError(f"{name} must be a contiguous {dtype} tensor of shape {list(shape)} on cuda:{idx}")


def _want(t, name, shape, dtype, idx):
    """t must be a contiguous tensor of this dtype and shape on CUDA device idx."""
    if t.dtype is not dtype or t.shape != shape or t.get_device() != idx or not t.is_contiguous():
        _refuse(name, shape, dtype, idx)


def _matrix(t, name, dtype):
    """Extents and device index of the matrix that a call's other tensors are held against."""
    if t.dtype is not dtype or t.dim() != 2 or not t.is_cuda or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous 2-D {dtype} CUDA tensor")
    rows, cols = t.shape
    return rows, cols, t.get_device()


def _word(t, name, idx):
    """The address of an optional one-element int32 tensor."""
    if t is None:
        return None
    if t.dtype is not _rd._torch().int32 or t.numel() != 1 or t.get_device() != idx:
        raise ValueError(f"{name} must be a one-element int32 tensor on cuda:{idx}")
    return t.data_ptr()


_current_device = _raw_stream = None


def _launch(fn, name, idx, device, stream, *args):
    """Call an entry point on the tensors' device, on its current stream or ``stream``."""
    global _current_device, _raw_stream
    if _current_device is None:
        torch = _rd._torch()
        # without the lazy-initialisation check of the public function, where it exists
        _current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
        _raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)
    if stream is None and _raw_stream is not None:
        handle = _raw_stream(idx)
    else:
        handle = _rd._stream(stream, device)
    if _current_device() == idx:
        code = fn(*args, handle)
    else:
        with _rd._on_device(device):
            code = fn(*args, handle)
    if code != 0:
        _rd._check(code, name)


def _used_on(stream, *outputs):
    """Outputs were allocated on the current stream and are written on ``stream`` (which the caller has
    ordered after the inputs): their memory is not handed out again before that work is done."""
    for t in outputs:
        t.record_stream(stream)


_configs = {}


def _config(*settings):
    """rd_route_config of these settings, by reference (one object for each set of settings)."""
    c = _configs.get(settings)
    if c is None:
        if len(_configs) >= 256:
            _configs.clear()
        c = _configs[settings] = ctypes.byref(_RouteConfig(*settings))
    return c


def _logits(logits):
    torch = _rd._torch()
    dtype = logits.dtype
    if dtype is torch.float32:
        return (_F32,) + _matrix(logits, "logits", dtype)
    if dtype is not torch.bfloat16:
        raise ValueError("logits must be float32 or bfloat16")
    return (_BF16,) + _matrix(logits, "logits", dtype)


def route(logits, topk: int, score: int = SCORE_SOFTMAX, bias=None, groups: int = 1,
          topk_groups: Optional[int] = None, renormalize: bool = True, scale: float = 1.0, limit=None,
          out: Optional[Routing] = None, stream=None) -> Routing:
    """Router logits [tokens, experts] to expert ids, weights and the packed buffer's plan (rd_route).

    ``topk_groups`` defaults to all groups.  ``out``: a Routing of buffers to write into.
    """
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    dtype, tokens, experts, idx = _logits(logits)
    dev, i32 = logits.device, torch.int32
    slots = (tokens, topk)
    if out is None:
        empty = torch.empty
        out = Routing(empty(slots, dtype=i32, device=dev), empty(slots, dtype=torch.float32, device=dev),
                      empty((experts,), dtype=i32, device=dev), empty(slots, dtype=i32, device=dev),
                      empty((1,), dtype=i32, device=dev))
    else:
        _want(out.ids, "ids", slots, i32, idx)
        _want(out.weights, "weights", slots, torch.float32, idx)
        _want(out.group_sizes, "group_sizes", (experts,), i32, idx)
        _want(out.pos, "pos", slots, i32, idx)
        _want(out.rows, "rows", (1,), i32, idx)
    bias_at = None
    if bias is not None:
        _want(bias, "bias", (experts,), torch.float32, idx)
        bias_at = bias.data_ptr()
    cfg = _config(topk, score, groups, groups if topk_groups is None else topk_groups,
                  1 if renormalize else 0, scale)
    ids, weights, sizes, pos, rows = out
    _launch(lib.rd_route, "rd_route", idx, dev, stream, logits.data_ptr(), dtype, bias_at, tokens,
            experts, cfg, _word(limit, "limit", idx), ids.data_ptr(), weights.data_ptr(), sizes.data_ptr(),
            pos.data_ptr(), rows.data_ptr())
    if stream is not None:
        _used_on(stream, *out)
    return out


def route_bwd(logits, ids, d_weights, score: int = SCORE_SOFTMAX, renormalize: bool = True,
              scale: float = 1.0, limit=None, out=None, stream=None):
    """Gradient of the logits from that of the weights (rd_route_bwd); settings as in ``route``."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    dtype, tokens, experts, idx = _logits(logits)
    topk = ids.shape[-1] if ids.dim() == 2 else 0
    _want(ids, "ids", (tokens, topk), torch.int32, idx)
    _want(d_weights, "d_weights", (tokens, topk), torch.float32, idx)
    if out is None:
        out = torch.empty_like(logits)
    else:
        _want(out, "out", (tokens, experts), logits.dtype, idx)
    cfg = _config(topk, score, 1, 1, 1 if renormalize else 0, scale)
    _launch(lib.rd_route_bwd, "rd_route_bwd", idx, logits.device, stream, logits.data_ptr(), dtype,
            ids.data_ptr(), d_weights.data_ptr(), tokens, experts, cfg, _word(limit, "limit", idx),
            out.data_ptr())
    if stream is not None:
        _used_on(stream, out)
    return out


def sort_rows(ids, experts: int, limit=None, stream=None):
    """(group_sizes [experts], pos [tokens, topk], rows [1]) of expert ids (rd_sort_rows)."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    i32 = torch.int32
    tokens, topk, idx = _matrix(ids, "ids", i32)
    dev = ids.device
    sizes = torch.empty((max(int(experts), 0),), dtype=i32, device=dev)
    pos = torch.empty_like(ids)
    rows = torch.empty((1,), dtype=i32, device=dev)
    _launch(lib.rd_sort_rows, "rd_sort_rows", idx, dev, stream, ids.data_ptr(), tokens, topk, int(experts),
            _word(limit, "limit", idx), sizes.data_ptr(), pos.data_ptr(), rows.data_ptr())
    if stream is not None:
        _used_on(stream, sizes, pos, rows)
    return sizes, pos, rows


def dispatch_rows(x, pos, out_rows: Optional[int] = None, limit=None, out=None, stream=None):
    """out[pos[t, k]] = x[t] (rd_dispatch_rows); out_rows defaults to tokens * topk."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    bf16 = torch.bfloat16
    tokens, hidden, idx = _matrix(x, "x", bf16)
    topk = pos.shape[-1] if pos.dim() == 2 else 0
    _want(pos, "pos", (tokens, topk), torch.int32, idx)
    if out_rows is None:
        out_rows = tokens * topk if out is None else out.shape[0]
    if out is None:
        out = torch.empty((out_rows, hidden), dtype=bf16, device=x.device)
    else:
        _want(out, "out", (out_rows, hidden), bf16, idx)
    _launch(lib.rd_dispatch_rows, "rd_dispatch_rows", idx, x.device, stream, x.data_ptr(), pos.data_ptr(),
            out.data_ptr(), tokens, topk, hidden, out_rows, _word(limit, "limit", idx))
    if stream is not None:
        _used_on(stream, out)
    return out


def combine_rows(y, pos, w=None, limit=None, out=None, stream=None):
    """out[t] = sum_k w[t, k] y[pos[t, k]] (rd_combine_rows); without ``w`` every weight is one."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    bf16 = torch.bfloat16
    rows, hidden, idx = _matrix(y, "y", bf16)
    tokens, topk = pos.shape if pos.dim() == 2 else (0, 0)
    _want(pos, "pos", (tokens, topk), torch.int32, idx)
    w_at = None
    if w is not None:
        _want(w, "w", (tokens, topk), torch.float32, idx)
        w_at = w.data_ptr()
    if out is None:
        out = torch.empty((tokens, hidden), dtype=bf16, device=y.device)
    else:
        _want(out, "out", (tokens, hidden), bf16, idx)
    _launch(lib.rd_combine_rows, "rd_combine_rows", idx, y.device, stream, y.data_ptr(), pos.data_ptr(),
            w_at, out.data_ptr(), tokens, topk, hidden, rows, _word(limit, "limit", idx))
    if stream is not None:
        _used_on(stream, out)
    return out


def combine_rows_bwd(d_out, y, pos, w, limit=None, d_y=None, d_w=None, stream=None):
    """(d_y, d_w) of ``combine_rows`` (rd_combine_rows_bwd)."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    bf16, f32 = torch.bfloat16, torch.float32
    rows, hidden, idx = _matrix(y, "y", bf16)
    tokens, topk = pos.shape if pos.dim() == 2 else (0, 0)
    _want(d_out, "d_out", (tokens, hidden), bf16, idx)
    _want(pos, "pos", (tokens, topk), torch.int32, idx)
    _want(w, "w", (tokens, topk), f32, idx)
    if d_y is None:
        d_y = torch.empty_like(y)
    else:
        _want(d_y, "d_y", (rows, hidden), bf16, idx)
    if d_w is None:
        d_w = torch.empty_like(w)
    else:
        _want(d_w, "d_w", (tokens, topk), f32, idx)
    _launch(lib.rd_combine_rows_bwd, "rd_combine_rows_bwd", idx, y.device, stream, d_out.data_ptr(),
            y.data_ptr(), pos.data_ptr(), w.data_ptr(), d_y.data_ptr(), d_w.data_ptr(), tokens, topk, hidden,
            rows, _word(limit, "limit", idx))
    if stream is not None:
        _used_on(stream, d_y, d_w)
    return d_y, d_w


def mxfp4_scale_width(k: int) -> int:
    """Bytes of one row's scales: k / 32 rounded up to a multiple of 16 (rd_mxfp4_scale_width)."""
    return 0 if k <= 0 else (k // 32 + 15) // 16 * 16


def mxfp4_quantize(x, pos=None, out_rows: Optional[int] = None, limit=None,
                   out: Optional[Mxfp4] = None, stream=None) -> Mxfp4:
    """bf16 rows [rows, k] to 4-bit rows; with ``pos`` straight to their packed rows (rd_mxfp4_quantize)."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    u8 = torch.uint8
    rows, k, idx = _matrix(x, "x", torch.bfloat16)
    topk, at = 1, None
    if pos is not None:
        topk = pos.shape[-1] if pos.dim() == 2 else 0
        _want(pos, "pos", (rows, topk), torch.int32, idx)
        at = pos.data_ptr()
    if out_rows is None:
        out_rows = rows * topk if out is None else out.q.shape[0]
    width = mxfp4_scale_width(k)
    if out is None:
        dev = x.device
        out = Mxfp4(torch.empty((out_rows, k // 2), dtype=u8, device=dev),
                    torch.empty((out_rows, width), dtype=u8, device=dev))
    else:
        _want(out.q, "q", (out_rows, k // 2), u8, idx)
        _want(out.scales, "scales", (out_rows, width), u8, idx)
    _launch(lib.rd_mxfp4_quantize, "rd_mxfp4_quantize", idx, x.device, stream, x.data_ptr(), at,
            out.q.data_ptr(), out.scales.data_ptr(), rows, topk, k, out_rows, _word(limit, "limit", idx))
    if stream is not None:
        _used_on(stream, *out)
    return out


def mxfp4_quantize_weights(rhs, out: Optional[Mxfp4] = None, stream=None) -> Mxfp4:
    """Expert weights [g, k, n] bf16 to 4-bit rows along k: q [g, n, k / 2] (rd_mxfp4_quantize_weights)."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    u8 = torch.uint8
    if rhs.dtype is not torch.bfloat16 or rhs.dim() != 3 or not rhs.is_cuda or not rhs.is_contiguous():
        raise ValueError("rhs must be a contiguous [g, k, n] bf16 CUDA tensor")
    g, k, n = rhs.shape
    idx, dev, width = rhs.get_device(), rhs.device, mxfp4_scale_width(k)
    if out is None:
        out = Mxfp4(torch.empty((g, n, k // 2), dtype=u8, device=dev),
                    torch.empty((g, n, width), dtype=u8, device=dev))
    else:
        _want(out.q, "q", (g, n, k // 2), u8, idx)
        _want(out.scales, "scales", (g, n, width), u8, idx)
    _launch(lib.rd_mxfp4_quantize_weights, "rd_mxfp4_quantize_weights", idx, dev, stream, rhs.data_ptr(),
            out.q.data_ptr(), out.scales.data_ptr(), g, k, n)
    if stream is not None:
        _used_on(stream, *out)
    return out


def mxfp4_dequantize(q, scales, limit=None, out=None, stream=None):
    """The values of 4-bit rows [rows, k / 2] as bf16 [rows, k] (rd_mxfp4_dequantize)."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    rows, half, idx = _matrix(q, "q", torch.uint8)
    k = 2 * half
    _want(scales, "scales", (rows, mxfp4_scale_width(k)), torch.uint8, idx)
    if out is None:
        out = torch.empty((rows, k), dtype=torch.bfloat16, device=q.device)
    else:
        _want(out, "out", (rows, k), torch.bfloat16, idx)
    _launch(lib.rd_mxfp4_dequantize, "rd_mxfp4_dequantize", idx, q.device, stream, q.data_ptr(),
            scales.data_ptr(), out.data_ptr(), rows, k, _word(limit, "limit", idx))
    if stream is not None:
        _used_on(stream, out)
    return out


def ragged_dot_mxfp4(a, a_scales, b, b_scales, group_sizes, group_offset: int = 0, limit=None,
                     epilogue: int = 0, out=None, out_scales=None, status=None, stream=None):
    """Grouped product of 4-bit rows a [m, k / 2] and weights b [g_local, n, k / 2] (rd_ragged_dot_mxfp4).

    EPI_NONE and EPI_SILU_GLU give bf16 rows, EPI_SILU_GLU_MXFP4 an Mxfp4 of 4-bit rows.
    """
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    u8 = torch.uint8
    m, half, idx = _matrix(a, "a", u8)
    if b.dim() != 3:
        raise ValueError("b must be [g_local, n, k / 2]")
    g_local, n, k = b.shape[0], b.shape[1], 2 * half
    width = mxfp4_scale_width(k)
    _want(b, "b", (g_local, n, half), u8, idx)
    _want(a_scales, "a_scales", (m, width), u8, idx)
    _want(b_scales, "b_scales", (g_local, n, width), u8, idx)
    g_total = group_sizes.numel()
    _want(group_sizes, "group_sizes", (g_total,), torch.int32, idx)
    quant = epilogue == EPI_SILU_GLU_MXFP4
    if quant:
        shape, dtype = (m, n // 4), u8
        scale_shape = (m, mxfp4_scale_width(n // 2))
        if out_scales is None:
            out_scales = torch.empty(scale_shape, dtype=u8, device=a.device)
        else:
            _want(out_scales, "out_scales", scale_shape, u8, idx)
    else:
        shape, dtype = (m, n // 2 if epilogue == _rd.EPI_SILU_GLU else n), torch.bfloat16
        if out_scales is not None:
            raise ValueError("out_scales belongs to EPI_SILU_GLU_MXFP4")
    if out is None:
        out = torch.empty(shape, dtype=dtype, device=a.device)
    else:
        _want(out, "out", shape, dtype, idx)
    _launch(lib.rd_ragged_dot_mxfp4, "rd_ragged_dot_mxfp4", idx, a.device, stream, a.data_ptr(),
            a_scales.data_ptr(), b.data_ptr(), b_scales.data_ptr(), out.data_ptr(),
            out_scales.data_ptr() if quant else None, m, k, n, group_sizes.data_ptr(), g_total,
            group_offset, g_local, _word(limit, "limit", idx), epilogue, _word(status, "status", idx))
    if stream is not None:
        _used_on(stream, *((out, out_scales) if quant else (out,)))
    return Mxfp4(out, out_scales) if quant else out
