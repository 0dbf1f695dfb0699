"""Python binding of the operators of a recurrent block (include/ssm2d_block.h):
linear projections with their epilogue, the norms before and after a block with
gate, residual and scale, and the gated linear recurrence.

Like the other bindings it only checks tensors and passes pointers, strides and
the HIP stream to libssm2d.so; every operator runs in the library's kernels.

    y = linear_fwd(x, weight, bias, residual, act="silu")       # rows, channels_first=True maps, or from one to the other
    g = linear_bwd(x, weight, dy, pre, act="silu")              # dict: dx, dweight, dbias
    out, y = block_norm_fwd(x, weight, gate=z, residual=r, next_weight=w2)
    g = block_norm_bwd(x, dout, dy, weight, gate=z, residual=r, next_weight=w2)   # dict: dx, dgate, dresidual, dweight, ...
    h = recurrence_fwd(x, g)                                    # sequences, packed with cu_seqlens=..., maps with channels_first
    g = recurrence_bwd(x, g, dh)                                # dict: dx, dg, dh_init
    h = recurrence_step(x, g, state)                            # one token, state updated in place

x, gates, weights of products and their gradients: float32 or bfloat16 (one type
in a call); biases, norms' weights, scales and states: float32. Inputs may be
strided views (the inner dim contiguous); outputs are dense, and take no part in
autograd: gradients come from the _bwd entries (examples/recurrent_block.py wraps
them). Workspaces are allocated for each call, from torch's allocator and on the
call's stream, so that calls may be captured into any number of graphs. Without
``stream`` a call runs on the current stream of its tensors' device; with one,
its outputs are allocated on that stream too, and ordering the inputs' producers
before it is the caller's.
"""
from __future__ import annotations

import ctypes
import functools

import torch

from . import OK, Ssm2dError, load_library
from .ops import _f32, _like, _new, _norm_layout, _on_gpu, _out, _ptr, _run

__all__ = ["linear_fwd", "linear_bwd", "block_norm_fwd", "block_norm_bwd", "recurrence_fwd", "recurrence_bwd", "recurrence_step"]

NORM_MAX_N = 16384
ACTS = {None: 0, "none": 0, "relu": 1, "silu": 2, "gelu": 3}
LINEAR_X_MAPS, LINEAR_Y_MAPS = 1, 2
NORM_ON, NORM_GATE_SIGMOID, NORM_GATE_FIRST, NORM_RESIDUAL_F32 = 1, 2, 4, 8
RECUR_SIGMOID, RECUR_MAPS, RECUR_REVERSE = 1, 2, 4

_vp, _i64, _u32 = ctypes.c_void_p, ctypes.c_int64, ctypes.c_uint32


class _LinearShape(ctypes.Structure):
    _fields_ = [("batch", _i64), ("rows", _i64), ("n", _i64), ("k", _i64), ("x_stride", _i64 * 2), ("r_stride", _i64 * 2), ("w_stride", _i64)]


class _NormShape(ctypes.Structure):
    _fields_ = [("rows", _i64), ("n", _i64), ("groups", _i64), ("x_stride", _i64), ("gate_stride", _i64), ("res_stride", _i64),
                ("dout_stride", _i64), ("dy_stride", _i64)]


class _RecurrenceShape(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64), ("channels", _i64), ("n_seq", _i64), ("x_stride", _i64 * 2), ("g_stride", _i64 * 2),
                ("dh_stride", _i64 * 2)]


def _p(struct):
    return ctypes.POINTER(struct)


_TAIL = [_vp, _i64, _vp]  # workspace, its bytes, stream
_SIGNATURES = {
    "ssm2d_linear_fwd": [_vp] * 6 + [_p(_LinearShape), ctypes.c_int, _u32] + _TAIL,
    "ssm2d_linear_bwd": [_vp] * 7 + [_p(_LinearShape), ctypes.c_int, _u32] + _TAIL,
    "ssm2d_block_norm_fwd": [_vp] * 8 + [_p(_NormShape), ctypes.c_float, _u32, _vp],
    "ssm2d_block_norm_bwd": [_vp] * 14 + [_p(_NormShape), ctypes.c_float, _u32] + _TAIL,
    "ssm2d_recurrence_fwd": [_vp] * 6 + [_p(_RecurrenceShape), _u32] + _TAIL,
    "ssm2d_recurrence_bwd": [_vp] * 9 + [_p(_RecurrenceShape), _u32] + _TAIL,
}
_WORKSPACES = {
    "ssm2d_linear_fwd_workspace": [_p(_LinearShape), _u32],
    "ssm2d_linear_bwd_workspace": [_p(_LinearShape), ctypes.c_int, _u32],
    "ssm2d_recurrence_fwd_workspace": [_p(_RecurrenceShape), _u32],
    "ssm2d_recurrence_bwd_workspace": [_p(_RecurrenceShape), _u32],
}
_PLAIN_WORKSPACES = {"ssm2d_block_norm_bwd_workspace": [_p(_NormShape), _u32]}  # (the same for both types)
_bound = {}


def _entry(name, dtype):
    """The C entry ``name`` for tensors of ``dtype`` (its _bf16 variant)."""
    f = _bound.get((name, dtype))
    if f is None:
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("tensors must be float32 or bfloat16")
        f = getattr(load_library(), name if dtype == torch.float32 or name in _PLAIN_WORKSPACES else name + "_bf16")
        f.argtypes = _SIGNATURES.get(name) or _WORKSPACES.get(name) or _PLAIN_WORKSPACES[name]
        f.restype = ctypes.c_int if name in _SIGNATURES else _i64
        _bound[name, dtype] = f
    return f


def _bytes(name, dtype, *args):
    """The workspace that a call of this shape needs."""
    n = _entry(name, dtype)(*args)
    if n < 0:
        raise Ssm2dError(-n, name)
    return n


def _workspace(n, dev, stream):
    return _new((n,), torch.uint8, dev, stream) if n else None


def _gpu(t, name="x"):
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16")
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    return t.device


# ------------------------------------------------------------------ linear

@functools.lru_cache(maxsize=256)
def _linear_shape(batch, rows, n, k, xs, rs, ws, dtype, act, flags, bwd):
    """(the C shape, the workspace's bytes)"""
    s = _LinearShape(batch, rows, n, k, xs, rs, ws)
    if bwd:
        return s, _bytes("ssm2d_linear_bwd_workspace", dtype, s, act, flags)
    return s, _bytes("ssm2d_linear_fwd_workspace", dtype, s, flags)


def _linear_layout(t, maps, by_batch, name):
    """(batch, rows, channels, (batch stride, row or channel stride)) of rows or maps."""
    if maps:
        b, c, cells, sb, sc = _norm_layout(t, True, name)
        return b, cells, c, (sb, sc)
    if by_batch:
        if t.dim() != 3:
            raise ValueError(f"{name} must be [batch, cells, channels]")
        if t.shape[2] > 1 and t.stride(2) != 1:
            raise ValueError(f"the channels of {name} must be contiguous")
        return t.shape[0], t.shape[1], t.shape[2], (t.stride(0), t.stride(1))
    rows, c, _, sr, _ = _norm_layout(t, False, name)
    return 1, rows, c, (0, sr)


def _linear(x, weight, act, channels_first, out_channels_first):
    """Checks shared by both directions: (device, act, flags, layout of x, n, weight's stride, shape of y, layout of a tensor like y)."""
    dev = _gpu(x)
    if act not in ACTS:
        raise ValueError(f"act must be one of {[a for a in ACTS if a]} or None")
    if out_channels_first is None:
        out_channels_first = channels_first
    if weight.dim() != 2 or weight.dtype != x.dtype:
        raise ValueError("weight must be [n, k] of x's dtype")
    if weight.shape[1] > 1 and weight.stride(1) != 1:
        raise ValueError("the rows of weight must be contiguous")
    mixed = channels_first or out_channels_first
    batch, rows, k, xs = _linear_layout(x, channels_first, mixed, "x")
    n = weight.shape[0]
    if weight.shape[1] != k:
        raise ValueError(f"x has {k} channels, weight takes {weight.shape[1]}")
    if channels_first:
        shape = (batch, n) + tuple(x.shape[2:]) if out_channels_first else (batch, rows, n)
    else:
        shape = (batch, n, rows) if out_channels_first else tuple(x.shape[:-1]) + (n,)
    flags = (LINEAR_X_MAPS if channels_first else 0) | (LINEAR_Y_MAPS if out_channels_first else 0)

    def like_y(t, name):
        if tuple(t.shape) != shape or t.dtype != x.dtype:
            raise ValueError(f"{name} must be {x.dtype} {list(shape)}")
        return _linear_layout(t, out_channels_first, mixed, name)[3]

    return dev, ACTS[act], flags, (batch, rows, k, xs), n, weight.stride(0), shape, like_y


def linear_fwd(x, weight, bias=None, residual=None, *, act=None, channels_first=False, out_channels_first=None, return_pre=False, y=None,
               stream=None):
    """y = act(x weight^T + bias) + residual. x: rows [..., k], or with
    ``channels_first`` maps [batch, k, ...] (the scan's layout); weight [n, k] of
    x's dtype, bias float32 [n]; act None, "relu", "silu" or "gelu" (by erf).
    ``out_channels_first`` (default: as x) lays y out the other way: from rows
    [batch, cells, k] to maps [batch, n, cells], or from maps to rows [batch,
    cells, n]. residual: y's shape and dtype. Returns y, or with ``return_pre``
    (y, pre): what act was applied to, for linear_bwd. ``y`` may be the residual."""
    dev, a, flags, (batch, rows, k, xs), n, ws, shape, like_y = _linear(x, weight, act, channels_first, out_channels_first)
    fn = _entry("ssm2d_linear_fwd", x.dtype)
    _on_gpu(dev, weight=weight, bias=bias, residual=residual)
    if bias is not None:
        _f32((n,), bias=bias)
    rs = like_y(residual, "residual") if residual is not None else (0, 0)
    s, need = _linear_shape(batch, rows, n, k, xs, rs, ws, x.dtype, a, flags, False)
    y = _out("y", y, shape, x.dtype, dev, stream)
    pre = _new(shape, x.dtype, dev, stream) if return_pre else None
    work = _workspace(need, dev, stream)
    _run(fn, dev, stream, (x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(pre), s, a, flags, _ptr(work), need))
    return (y, pre) if return_pre else y


def linear_bwd(x, weight, dy, pre=None, *, act=None, bias=True, channels_first=False, out_channels_first=None, out=None, stream=None):
    """Gradients of linear_fwd for dy, with the pre that it returned (needed with
    an activation): a dict dx, dweight (x's dtype) and, with ``bias``, dbias (float32
    [n]). The residual's gradient is dy. ``out`` may supply any of them."""
    dev, a, flags, (batch, rows, k, xs), n, ws, shape, like_y = _linear(x, weight, act, channels_first, out_channels_first)
    fn = _entry("ssm2d_linear_bwd", x.dtype)
    _on_gpu(dev, weight=weight, dy=dy, pre=pre)
    rs = like_y(dy, "dy")
    if a:
        if pre is None:
            raise ValueError("pre is required with an activation")
        if tuple(pre.shape) != shape or pre.dtype != x.dtype or not pre.is_contiguous():
            raise ValueError(f"pre must be contiguous {x.dtype} {list(shape)}")
    out = out or {}
    r = {"dx": _out("dx", out.get("dx"), tuple(x.shape), x.dtype, dev, stream),
         "dweight": _out("dweight", out.get("dweight"), (n, k), x.dtype, dev, stream)}
    if bias:
        r["dbias"] = _out("dbias", out.get("dbias"), (n,), torch.float32, dev, stream)
    s, need = _linear_shape(batch, rows, n, k, xs, rs, ws, x.dtype, a, flags, True)
    work = _workspace(need, dev, stream)
    _run(fn, dev, stream, (x.data_ptr(), weight.data_ptr(), _ptr(pre) if a else None, dy.data_ptr(), r["dx"].data_ptr(), r["dweight"].data_ptr(),
                           _ptr(r.get("dbias")), s, a, flags, _ptr(work), need))
    return r


# ------------------------------------------------------------------ block norm

@functools.lru_cache(maxsize=256)
def _norm_shape(rows, n, groups, xs, gs, rs, os, ys, flags, bwd):
    s = _NormShape(rows, n, groups, xs, gs, rs, os, ys)
    return s, _bytes("ssm2d_block_norm_bwd_workspace", torch.float32, s, flags) if bwd else 0


def _rows_like(t, x, name, dtypes):
    """The row stride of an optional tensor of x's shape."""
    if t is None:
        return 0
    if t.shape != x.shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must have x's shape, and {' or '.join(map(str, dtypes))}")
    return _norm_layout(t, False, name)[3]


def _block_norm(x, weight, gate, residual, scale, next_weight, norm, groups, gate_act, gate_first):
    dev = _gpu(x)
    rows, n, _, xs, _ = _norm_layout(x, False)
    if not 0 < groups or n % groups:
        raise ValueError("the channels must be a multiple of groups")
    if gate_act not in ("silu", "sigmoid"):
        raise ValueError('gate_act must be "silu" or "sigmoid"')
    if weight is not None and not norm:
        raise ValueError("weight belongs to the norm")
    _on_gpu(dev, weight=weight, gate=gate, residual=residual, scale=scale, next_weight=next_weight)
    _f32((n,), weight=weight, scale=scale, next_weight=next_weight)
    gs = _rows_like(gate, x, "gate", (x.dtype,))
    rs = _rows_like(residual, x, "residual", (x.dtype, torch.float32) if x.dtype != torch.float32 else (x.dtype,))
    flags = (NORM_ON if norm else 0) | (NORM_GATE_SIGMOID if gate_act == "sigmoid" else 0) | (NORM_GATE_FIRST if gate_first else 0)
    return dev, rows, n, xs, gs, rs, flags


def block_norm_fwd(x, weight=None, *, gate=None, residual=None, scale=None, next_weight=None, norm=True, groups=1, gate_act="silu",
                   gate_first=False, eps=1e-5, out_dtype=None, out=None, y=None, stream=None):
    """The norm after a block, its gate, scale and residual, and the norm before
    the next one, over the last dim of x [..., n]:
        m = rms(x) weight act(gate)    (gate_first: rms(x act(gate)) weight)
        out = residual + scale m
        y = rms(out) next_weight       (with next_weight only)
    where rms divides by the root of the mean square + eps, the first one over
    ``groups`` equal groups of channels each by itself; ``norm=False`` leaves it
    out. gate: x's shape and dtype; residual: x's shape, its dtype or float32;
    weight, scale, next_weight: float32 [n]; all but x may be None. out has the
    residual's dtype (``out_dtype``, x's dtype or float32, where there is none).
    Returns out, or (out, y) with next_weight. ``out`` may be the residual."""
    dev, rows, n, xs, gs, rs, flags = _block_norm(x, weight, gate, residual, scale, next_weight, norm, groups, gate_act, gate_first)
    fn = _entry("ssm2d_block_norm_fwd", x.dtype)
    if out_dtype is None:
        out_dtype = residual.dtype if residual is not None else x.dtype
    elif out_dtype not in (x.dtype, torch.float32) or (residual is not None and out_dtype != residual.dtype):
        raise ValueError("out_dtype must be the residual's dtype, or x's or float32 without one")
    if out_dtype != x.dtype:
        flags |= NORM_RESIDUAL_F32
    out = _out("out", out, x.shape, out_dtype, dev, stream)
    if next_weight is not None:
        y = _out("y", y, x.shape, x.dtype, dev, stream)
    elif y is not None:
        raise ValueError("y needs next_weight")
    s, _ = _norm_shape(rows, n, groups, xs, gs, rs, 0, 0, flags, False)
    _run(fn, dev, stream, (x.data_ptr(), _ptr(gate), _ptr(residual), _ptr(weight), _ptr(scale), _ptr(next_weight), out.data_ptr(), _ptr(y), s,
                           float(eps), flags))
    return (out, y) if next_weight is not None else out


def block_norm_bwd(x, dout, dy=None, weight=None, *, gate=None, residual=None, scale=None, next_weight=None, norm=True, groups=1,
                   gate_act="silu", gate_first=False, eps=1e-5, out=None, stream=None):
    """Gradients of block_norm_fwd for dout (the gradient that reaches out
    otherwise than through y, of out's dtype; None: none) and, with next_weight,
    dy (None: none): a dict of dx and, of what was given, dgate, dresidual, and
    dweight, dscale, dnext_weight (float32 [n]). Nothing of the forward but its
    inputs is needed. ``out`` may supply any of them."""
    dev, rows, n, xs, gs, rs, flags = _block_norm(x, weight, gate, residual, scale, next_weight, norm, groups, gate_act, gate_first)
    fn = _entry("ssm2d_block_norm_bwd", x.dtype)
    if dy is not None and next_weight is None:
        raise ValueError("dy needs next_weight")
    if dout is None and dy is None:
        raise ValueError("dout or dy is required")
    rt = residual.dtype if residual is not None else (dout.dtype if dout is not None else x.dtype)
    _on_gpu(dev, dout=dout, dy=dy)
    if rt not in (x.dtype, torch.float32):
        raise ValueError("dout must have out's dtype")
    os, ys = _rows_like(dout, x, "dout", (rt,)), _rows_like(dy, x, "dy", (x.dtype,))
    if rt != x.dtype:
        flags |= NORM_RESIDUAL_F32
    out, r = out or {}, {}

    def result(name, given, shape, dtype):
        if given is not None:
            r[name] = _out(name, out.get(name), shape, dtype, dev, stream)

    result("dx", x, x.shape, x.dtype)
    result("dgate", gate, x.shape, x.dtype)
    result("dresidual", residual, x.shape, rt)
    result("dweight", weight, (n,), torch.float32)
    result("dscale", scale, (n,), torch.float32)
    result("dnext_weight", next_weight, (n,), torch.float32)
    s, need = _norm_shape(rows, n, groups, xs, gs, rs, os, ys, flags, True)
    work = _workspace(need, dev, stream)
    _run(fn, dev, stream, (x.data_ptr(), _ptr(gate), _ptr(residual), _ptr(weight), _ptr(scale), _ptr(next_weight), _ptr(dout), _ptr(dy),
                           r["dx"].data_ptr(), *(_ptr(r.get(k)) for k in ("dgate", "dresidual", "dweight", "dscale", "dnext_weight")), s,
                           float(eps), flags, _ptr(work), need))
    return r


# ------------------------------------------------------------------ recurrence

@functools.lru_cache(maxsize=256)
def _recurrence_shape(batch, tokens, channels, n_seq, xs, gs, ds, dtype, flags, bwd):
    s = _RecurrenceShape(batch, tokens, channels, n_seq, xs, gs, ds)
    return s, _bytes("ssm2d_recurrence_bwd_workspace" if bwd else "ssm2d_recurrence_fwd_workspace", dtype, s, flags)


def _sequence_layout(t, maps, name):
    """(batch, tokens, channels, (batch stride, token or channel stride))"""
    if maps:
        b, c, tokens, sb, sc = _norm_layout(t, True, name)
        return b, tokens, c, (sb, sc)
    return _linear_layout(t, False, True, name)


def _recurrence(x, g, gates, cu_seqlens, channels_first, reverse, dh=None):
    dev = _gpu(x)
    if gates not in ("decay", "sigmoid"):
        raise ValueError('gates must be "decay" or "sigmoid"')
    if g.shape != x.shape or g.dtype != x.dtype:
        raise ValueError("g must match x in shape and dtype")
    batch, tokens, channels, xs = _sequence_layout(x, channels_first, "x")
    gs = _sequence_layout(g, channels_first, "g")[3]
    ds = (0, 0)
    if dh is not None:
        if dh.shape != x.shape or dh.dtype != x.dtype:
            raise ValueError("dh must match x in shape and dtype")
        ds = _sequence_layout(dh, channels_first, "dh")[3]
    n_seq = 0
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous int32 [sequences + 1], at least one sequence")
        if batch != 1 or channels_first or reverse:
            raise ValueError("packed sequences need batch 1, and go neither channels first nor in reverse")
        n_seq = cu_seqlens.numel() - 1
    _on_gpu(dev, g=g, cu_seqlens=cu_seqlens, dh=dh)
    flags = (RECUR_SIGMOID if gates == "sigmoid" else 0) | (RECUR_MAPS if channels_first else 0) | (RECUR_REVERSE if reverse else 0)
    return dev, flags, (n_seq or batch, channels), _recurrence_shape(batch, tokens, channels, n_seq, xs, gs, ds, x.dtype, flags, dh is not None)


def recurrence_fwd(x, g, *, gates="decay", h_init=None, cu_seqlens=None, channels_first=False, reverse=False, return_last_state=False, h=None,
                   h_last=None, stream=None):
    """h[t] = a[t] h[t - 1] + w[t] x[t] of each channel along the tokens: a =
    exp(g), w = 1 with ``gates`` "decay" (g the log decay), a = sigmoid(g), w = 1 - a
    with "sigmoid". x, g: [batch, tokens, channels], or with ``channels_first``
    [batch, channels, ...] with the cells as tokens; ``reverse`` goes from the last
    token to the first. With ``cu_seqlens`` (int32 [sequences + 1], batch 1) the
    tokens hold packed sequences; tokens behind the last one are left as they
    were. h_init: float32 [sequences, channels] or None (zeros). Returns h (x's
    shape and dtype), or (h, h_last)."""
    dev, flags, states, (shape, need) = _recurrence(x, g, gates, cu_seqlens, channels_first, reverse)
    fn = _entry("ssm2d_recurrence_fwd", x.dtype)
    _on_gpu(dev, h_init=h_init)
    _f32(states, h_init=h_init)
    h = _like("h", h, x, stream)
    if return_last_state or h_last is not None:
        h_last = _out("h_last", h_last, states, torch.float32, dev, stream)
    work = _workspace(need, dev, stream)
    _run(fn, dev, stream, (x.data_ptr(), g.data_ptr(), _ptr(h_init), _ptr(cu_seqlens), h.data_ptr(), _ptr(h_last), shape, flags, _ptr(work), need))
    return (h, h_last) if return_last_state else h


def recurrence_bwd(x, g, dh, *, gates="decay", h_init=None, dh_last=None, cu_seqlens=None, channels_first=False, reverse=False, out=None,
                   stream=None):
    """Gradients of recurrence_fwd for dh = dL/dh and dh_last = dL/dh_last (None:
    zeros): a dict dx, dg (x's dtype), and dh_init (float32) when h_init or
    dh_last is given or ``out`` holds it. ``out`` may supply any of them."""
    dev, flags, states, (shape, need) = _recurrence(x, g, gates, cu_seqlens, channels_first, reverse, dh)
    fn = _entry("ssm2d_recurrence_bwd", x.dtype)
    _on_gpu(dev, h_init=h_init, dh_last=dh_last)
    _f32(states, h_init=h_init, dh_last=dh_last)
    out = out or {}
    r = {n: _like(n, out.get(n), x, stream) for n in ("dx", "dg")}
    if h_init is not None or dh_last is not None or out.get("dh_init") is not None:
        r["dh_init"] = _out("dh_init", out.get("dh_init"), states, torch.float32, dev, stream)
    work = _workspace(need, dev, stream)
    _run(fn, dev, stream, (x.data_ptr(), g.data_ptr(), _ptr(h_init), _ptr(cu_seqlens), dh.data_ptr(), _ptr(dh_last), r["dx"].data_ptr(),
                           r["dg"].data_ptr(), _ptr(r.get("dh_init")), shape, flags, _ptr(work), need))
    return r


def recurrence_step(x, g, state, *, gates="decay", h=None, stream=None):
    """One token of the recurrence for each batch entry: x, g [batch, channels];
    state: float32 [batch, channels], updated in place. Returns h (x's shape and
    dtype)."""
    if x.dim() != 2:
        raise ValueError("x and g must be [batch, channels]")
    if state is None:
        raise ValueError("state is required")
    dev = _gpu(x)
    batch, channels = x.shape
    if gates not in ("decay", "sigmoid"):
        raise ValueError('gates must be "decay" or "sigmoid"')
    if g.shape != x.shape or g.dtype != x.dtype:
        raise ValueError("g must match x in shape and dtype")
    if channels > 1 and (x.stride(1) != 1 or g.stride(1) != 1):
        raise ValueError("the channels of x and g must be contiguous")
    fn = _entry("ssm2d_recurrence_fwd", x.dtype)
    _on_gpu(dev, g=g, state=state)
    _f32((batch, channels), state=state)
    flags = RECUR_SIGMOID if gates == "sigmoid" else 0
    shape, need = _recurrence_shape(batch, 1, channels, 0, (x.stride(0), 0), (g.stride(0), 0), (0, 0), x.dtype, flags, False)
    h = _like("h", h, x, stream)
    work = _workspace(need, dev, stream)
    _run(fn, dev, stream, (x.data_ptr(), g.data_ptr(), state.data_ptr(), None, h.data_ptr(), state.data_ptr(), shape, flags, _ptr(work), need))
    return h
