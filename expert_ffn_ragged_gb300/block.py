"""Binding of include/rd_block.h: the rest of a feed-forward block around the experts.

Argument marshalling only, as in the package itself (whose functions these are, too):

* ``layer_norm_fwd(x, weight, bias, ...)``             -> LayerNorm(out, mean, rstd)
* ``layer_norm_bwd(d_out, x, weight, mean, rstd, ...)`` -> (d_x, d_weight, d_bias)
* ``linear(x, w, bias, residual, act, ...)``           -> out, or (out, pre)
* ``linear_act_bwd(d_out, pre, act, ...)``             -> (d_pre, d_bias)
* ``dropout_rows(x, rng, p, residual, ...)``           -> out; its gradient is the same call on the
  gradient of out, without a residual

A block: ``layer_norm_fwd`` the tokens, ``linear`` them to router logits (f32), run the experts (or two
``linear`` calls, activation in the first, residual in the second), ``dropout_rows`` the result onto
the residual stream.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Optional

import expert_ffn_ragged_gb300 as _rd

from .moe import _launch, _matrix, _used_on, _want, _word

ACT_NONE = 0
ACT_RELU = 1
ACT_GELU = 2
ACT_GELU_TANH = 3
ACT_SILU = 4

_F32, _BF16 = 0, 1


class LayerNorm(NamedTuple):
    """What ``layer_norm_fwd`` gives: out [rows, hidden]; mean and rstd [rows] f32, or None."""

    out: object
    mean: object
    rstd: object


def declare(lib):
    """Argument and result types of the entry points of rd_block.h."""
    vp, i64, i32, f32, sz = (ctypes.c_void_p, ctypes.c_int64, ctypes.c_int32, ctypes.c_float, ctypes.c_size_t)
    for name, args in (
            ("rd_layer_norm_fwd", [vp, i32, vp, vp, f32, vp, i32, vp, vp, i64, i64, vp, vp]),
            ("rd_layer_norm_bwd", [vp, i32, vp, i32, vp, vp, vp, vp, vp, vp, i64, i64, vp, vp, sz, vp]),
            ("rd_layer_norm_bwd_workspace_size", [i64, i64, vp]),
            ("rd_linear", [vp, vp, vp, vp, i32, vp, i32, vp, i64, i64, i64, vp, i32, i32, i32, vp, vp, vp]),
            ("rd_linear_act_bwd", [vp, i32, vp, i32, vp, vp, i64, i64, vp, i32, i32, i32, vp, vp, sz, vp, vp]),
            ("rd_linear_act_bwd_workspace_size", [i64, i64, i32, vp]),
            ("rd_dropout_rows", [vp, i32, vp, vp, f32, vp, i32, i64, i64, vp, vp])):
        fn = getattr(lib, name)
        fn.argtypes = args
        fn.restype = ctypes.c_int


def _typed(t, name):
    """Type number, extents and device index of a matrix of f32 or bf16."""
    torch = _rd._torch()
    dtype = t.dtype
    if dtype is torch.bfloat16:
        return (_BF16,) + _matrix(t, name, dtype)
    if dtype is not torch.float32:
        raise ValueError(f"{name} must be float32 or bfloat16")
    return (_F32,) + _matrix(t, name, dtype)


def _type_of(dtype, name):
    torch = _rd._torch()
    if dtype is torch.bfloat16:
        return _BF16
    if dtype is torch.float32:
        return _F32
    raise ValueError(f"{name} must be torch.float32 or torch.bfloat16")


def _vector(t, name, shape, idx):
    """The address of an optional f32 parameter of this shape."""
    if t is None:
        return None
    _want(t, name, shape, _rd._torch().float32, idx)
    return t.data_ptr()


def _at(t):
    return None if t is None else t.data_ptr()


def layer_norm_fwd(x, weight=None, bias=None, eps: float = 1e-5, limit=None, out_dtype=None,
                   stats: bool = True, out: Optional[LayerNorm] = None, stream=None) -> LayerNorm:
    """Layer norm of rows [rows, hidden] (rd_layer_norm_fwd), in ``out_dtype`` (default: that of x).

    ``stats`` keeps the rows' mean and 1 / deviation, which ``layer_norm_bwd`` reads.
    ``out``: a LayerNorm of buffers to write into (its statistics may be None, its type rules).
    """
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    dtype, rows, hidden, idx = _typed(x, "x")
    dev, f32 = x.device, torch.float32
    if out is None:
        y = torch.empty((rows, hidden), dtype=x.dtype if out_dtype is None else out_dtype, device=dev)
        out_type = _type_of(y.dtype, "out_dtype")
        mean = rstd = None
        if stats:
            mean, rstd = torch.empty((rows,), dtype=f32, device=dev), torch.empty((rows,), dtype=f32, device=dev)
        out = LayerNorm(y, mean, rstd)
    else:
        y, mean, rstd = out
        out_type = _type_of(y.dtype if out_dtype is None else out_dtype, "out_dtype")
        _want(y, "out", (rows, hidden), torch.bfloat16 if out_type == _BF16 else f32, idx)
        if (mean is None) != (rstd is None):
            raise ValueError("mean and rstd come together")
    w_at, b_at = _vector(weight, "weight", (hidden,), idx), _vector(bias, "bias", (hidden,), idx)
    _launch(lib.rd_layer_norm_fwd, "rd_layer_norm_fwd", idx, dev, stream, x.data_ptr(), dtype, w_at, b_at, eps,
            y.data_ptr(), out_type, _vector(mean, "mean", (rows,), idx), _vector(rstd, "rstd", (rows,), idx), rows,
            hidden, _word(limit, "limit", idx))
    if stream is not None:
        _used_on(stream, *(t for t in out if t is not None))
    return out


_norm_bytes = {}


def layer_norm_bwd_workspace_bytes(rows: int, hidden: int, device=None) -> int:
    """Bytes of the workspace of ``layer_norm_bwd`` (rd_layer_norm_bwd_workspace_size)."""
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    n = ctypes.c_size_t(0)
    with _rd._on_device(dev):
        _rd._check(lib.rd_layer_norm_bwd_workspace_size(rows, hidden, ctypes.byref(n)),
                   "rd_layer_norm_bwd_workspace_size")
    return n.value


def linear_act_bwd_workspace_bytes(m: int, n: int, g_local: int = 1) -> int:
    """Bytes of the workspace of ``linear_act_bwd`` (rd_linear_act_bwd_workspace_size)."""
    lib = _rd._lib or _rd.load()
    size = ctypes.c_size_t(0)
    _rd._check(lib.rd_linear_act_bwd_workspace_size(m, n, g_local, ctypes.byref(size)),
               "rd_linear_act_bwd_workspace_size")
    return size.value


def _scratch(workspace, need, dev, idx):
    """The caller's workspace, or one of the needed size."""
    torch = _rd._torch()
    if workspace is None:
        return torch.empty((need,), dtype=torch.uint8, device=dev)
    if (workspace.dtype is not torch.uint8 or workspace.get_device() != idx or not workspace.is_contiguous()):
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{idx}")
    return workspace


def layer_norm_bwd(d_out, x, weight, mean, rstd, limit=None, need_weight: bool = True, need_bias: bool = True,
                   d_x=None, d_weight=None, d_bias=None, workspace=None, stream=None):
    """(d_x, d_weight, d_bias) of ``layer_norm_fwd`` (rd_layer_norm_bwd); None where not needed.

    ``workspace``: a uint8 tensor of ``layer_norm_bwd_workspace_bytes``; by default a new one.
    """
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    f32 = torch.float32
    dtype, rows, hidden, idx = _typed(x, "x")
    out_type = _type_of(d_out.dtype, "d_out's type")
    _want(d_out, "d_out", (rows, hidden), d_out.dtype, idx)
    _want(mean, "mean", (rows,), f32, idx)
    _want(rstd, "rstd", (rows,), f32, idx)
    w_at = _vector(weight, "weight", (hidden,), idx)
    dev = x.device
    if d_x is None:
        d_x = torch.empty_like(x)
    else:
        _want(d_x, "d_x", (rows, hidden), x.dtype, idx)
    if d_weight is None and need_weight:
        d_weight = torch.empty((hidden,), dtype=f32, device=dev)
    if d_bias is None and need_bias:
        d_bias = torch.empty((hidden,), dtype=f32, device=dev)
    dw_at, db_at = _vector(d_weight, "d_weight", (hidden,), idx), _vector(d_bias, "d_bias", (hidden,), idx)
    scratch = None
    if d_weight is not None or d_bias is not None:
        key = (idx, rows, hidden)
        need = _norm_bytes.get(key)
        if need is None:
            if len(_norm_bytes) >= 1024:
                _norm_bytes.clear()
            need = _norm_bytes[key] = layer_norm_bwd_workspace_bytes(rows, hidden, dev)
        scratch = workspace
        if workspace is not None or need:
            scratch = _scratch(workspace, need, dev, idx)
    _launch(lib.rd_layer_norm_bwd, "rd_layer_norm_bwd", idx, dev, stream, d_out.data_ptr(), out_type, x.data_ptr(),
            dtype, w_at, mean.data_ptr(), rstd.data_ptr(), d_x.data_ptr(), dw_at, db_at, rows, hidden,
            _word(limit, "limit", idx), _at(scratch), 0 if scratch is None else scratch.numel())
    if stream is not None:
        _used_on(stream, *(t for t in (d_x, d_weight, d_bias, scratch) if t is not None))
    return d_x, d_weight, d_bias


_act_sizes = {}


def _act_bytes(m, n, g_local):
    """linear_act_bwd_workspace_bytes, asked once for each set of sizes."""
    key = (m, n, g_local)
    need = _act_sizes.get(key)
    if need is None:
        if len(_act_sizes) >= 1024:
            _act_sizes.clear()
        need = _act_sizes[key] = linear_act_bwd_workspace_bytes(m, n, g_local)
    return need


def _groups(group_sizes, idx):
    """(address, g_total) of optional group sizes."""
    if group_sizes is None:
        return None, 1
    g_total = group_sizes.numel()
    _want(group_sizes, "group_sizes", (g_total,), _rd._torch().int32, idx)
    return group_sizes.data_ptr(), g_total


def linear(x, w, bias=None, residual=None, act: int = ACT_NONE, group_sizes=None, group_offset: int = 0,
           limit=None, out_dtype=None, save_pre: bool = False, out=None, pre=None, status=None, stream=None):
    """act(x @ w + bias) + residual (rd_linear); x [m, k] bf16, in ``out_dtype`` (default bfloat16).

    One weight: w [k, n], bias [n].  By expert: w [g_local, k, n], bias [g_local, n] and
    ``group_sizes``.  ``save_pre`` (or a ``pre`` buffer) also keeps the rows before the activation, as bf16,
    for ``linear_act_bwd``: the result is then (out, pre).
    """
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    bf16 = torch.bfloat16
    m, k, idx = _matrix(x, "x", bf16)
    if group_sizes is None:
        if w.dim() != 2 or group_offset != 0:
            raise ValueError("without group_sizes, w must be [k, n] and group_offset 0")
        n, g_local = w.shape[1], 1
        _want(w, "w", (k, n), bf16, idx)
        b_at = _vector(bias, "bias", (n,), idx)
    else:
        if w.dim() != 3:
            raise ValueError("with group_sizes, w must be [g_local, k, n]")
        g_local, n = w.shape[0], w.shape[2]
        _want(w, "w", (g_local, k, n), bf16, idx)
        b_at = _vector(bias, "bias", (g_local, n), idx)
    sizes_at, g_total = _groups(group_sizes, idx)
    dev, shape = x.device, (m, n)
    if out is None:
        dtype = bf16 if out_dtype is None else out_dtype
        out_type = _type_of(dtype, "out_dtype")
        out = torch.empty(shape, dtype=dtype, device=dev)
    else:
        dtype = out.dtype if out_dtype is None else out_dtype
        out_type = _type_of(dtype, "out_dtype")
        _want(out, "out", shape, dtype, idx)
    if residual is not None:
        _want(residual, "residual", shape, dtype, idx)
    if pre is not None:
        _want(pre, "pre", shape, bf16, idx)
    elif save_pre:
        pre = torch.empty(shape, dtype=bf16, device=dev)
    _launch(lib.rd_linear, "rd_linear", idx, dev, stream, x.data_ptr(), w.data_ptr(), b_at, _at(residual), act,
            out.data_ptr(), out_type, _at(pre), m, k, n, sizes_at, g_total, group_offset, g_local,
            _word(limit, "limit", idx), _word(status, "status", idx))
    if stream is not None:
        _used_on(stream, *((out,) if pre is None else (out, pre)))
    return out if pre is None else (out, pre)


def linear_act_bwd(d_out, pre, act: int = ACT_NONE, group_sizes=None, group_offset: int = 0,
                   g_local: Optional[int] = None, limit=None, need_pre: bool = True, need_bias: bool = True,
                   d_pre=None, d_bias=None, workspace=None, status=None, stream=None):
    """(d_pre, d_bias) of ``linear`` in front of its activation (rd_linear_act_bwd); None where not needed.

    d_out [m, n] f32 or bf16, pre [m, n] bf16 (None with ACT_NONE).  d_bias is [n], or
    [g_local, n] with ``group_sizes`` (g_local defaults to the groups from group_offset on).
    ``workspace``: a uint8 tensor of ``linear_act_bwd_workspace_bytes``; by default a new one.
    """
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    bf16, f32 = torch.bfloat16, torch.float32
    out_type, m, n, idx = _typed(d_out, "d_out")
    if pre is not None:
        _want(pre, "pre", (m, n), bf16, idx)
    sizes_at, g_total = _groups(group_sizes, idx)
    if g_local is None:
        g_local = g_total - group_offset
    dev = d_out.device
    shape = (n,) if group_sizes is None else (max(g_local, 0), n)
    if d_pre is not None:
        _want(d_pre, "d_pre", (m, n), bf16, idx)
    elif need_pre:
        d_pre = torch.empty((m, n), dtype=bf16, device=dev)
    if d_bias is not None:
        _want(d_bias, "d_bias", shape, f32, idx)
    elif need_bias:
        d_bias = torch.empty(shape, dtype=f32, device=dev)
    scratch = workspace
    if d_bias is not None and g_local >= 1:
        need = 0 if workspace is not None else _act_bytes(m, n, g_local)
        if workspace is not None or need:
            scratch = _scratch(workspace, need, dev, idx)
    _launch(lib.rd_linear_act_bwd, "rd_linear_act_bwd", idx, dev, stream, d_out.data_ptr(), out_type, _at(pre), act,
            _at(d_pre), _at(d_bias), m, n, sizes_at, g_total, group_offset, g_local, _word(limit, "limit", idx),
            _at(scratch), 0 if scratch is None else scratch.numel(), _word(status, "status", idx))
    if stream is not None:
        _used_on(stream, *(t for t in (d_pre, d_bias, scratch) if t is not None))
    return d_pre, d_bias


def dropout_rows(x, rng, p: float, residual=None, limit=None, out_dtype=None, out=None, stream=None):
    """Dropout of rows [rows, hidden] with the generator's words ``rng`` (int64 [2]: a seed and an offset, on
    the device), plus ``residual`` (rd_dropout_rows), in ``out_dtype`` (default: that of the residual, else of x).
    """
    torch = _rd._torch()
    lib = _rd._lib or _rd.load()
    dtype, rows, hidden, idx = _typed(x, "x")
    _want(rng, "rng", (2,), torch.int64, idx)
    if out is not None:
        kind = out.dtype if out_dtype is None else out_dtype
        out_type = _type_of(kind, "out_dtype")
        _want(out, "out", (rows, hidden), kind, idx)
    else:
        kind = out_dtype if out_dtype is not None else (x if residual is None else residual).dtype
        out_type = _type_of(kind, "out_dtype")
        out = torch.empty((rows, hidden), dtype=kind, device=x.device)
    if residual is not None:
        _want(residual, "residual", (rows, hidden), kind, idx)
    _launch(lib.rd_dropout_rows, "rd_dropout_rows", idx, x.device, stream, x.data_ptr(), dtype, _at(residual),
            rng.data_ptr(), p, out.data_ptr(), out_type, rows, hidden, _word(limit, "limit", idx))
    if stream is not None:
        _used_on(stream, out)
    return out
