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
strided views (the inner dim contiguous); outputs are dense, share no memory with
an input unless it is said so, and take no part in
autograd: gradients come from the _bwd entries (examples/recurrent_block.py wraps
them). Workspaces are allocated for each call, from torch's allocator and on the
call's stream, so that calls may be captured into any number of graphs. Without
``stream`` a call runs on the current stream of its tensors' device; with one,
its outputs are allocated on that stream too, and ordering the inputs' producers
before it is the caller's.
"""
from __future__ import annotations

import ctypes
import operator

import torch

from . import ERR_HIP, OK, Ssm2dError, load_library
from .ops import _f32, _new, _norm_layout, _on_gpu, _out, _raw_stream

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


def _gpu(t, name="x"):
    if t.dtype not in (torch.float32, torch.bfloat16):
        raise TypeError(f"{name} must be float32 or bfloat16")
    if t.device.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    return t.device


# What a call's checks come to depends on its tensors' shapes, strides, types and
# devices alone: it is kept by those, and the next call of the kind pays for
# reading them (half of one token's call otherwise: 12 of 22 us of host time).
_plans = {}


def _meta(t):
    return None if t is None else (t.shape, t.stride(), t.dtype, t.get_device())


def _keep(key, plan):
    if len(_plans) >= 4096:
        _plans.clear()
    _plans[key] = plan
    return plan


_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


def _launch(fn, index, stream, args):
    """Calls fn(*args, stream) with device ``index`` current; a status becomes an exception."""
    handle = stream.cuda_stream if stream is not None else _raw_stream(index)
    if _current_device() == index:
        s = fn(*args, handle)
    else:
        with torch.cuda.device(index):
            s = fn(*args, handle)
    if s != OK:
        raise Ssm2dError(s, fn.__name__ + (f" ({load_library().ssm2d_last_hip_error().decode()})" if s == ERR_HIP else ""))


def _make(name, t, shape, dtype, like, stream):
    """An output: given, or allocated on the device of ``like``."""
    if t is None and stream is None:
        return torch.empty_like(like) if dtype is like.dtype and like.shape == shape and like.is_contiguous() else like.new_empty(shape, dtype=dtype)
    return _out(name, t, shape, dtype, like.device, stream)


def _workspace(n, like, stream):
    if not n:
        return None
    return like.new_empty(n, dtype=torch.uint8) if stream is None else _new((n,), torch.uint8, like.device, stream)


def _ptr(t):
    return None if t is None else t.data_ptr()


# ------------------------------------------------------------------ linear

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


def _act(act):
    if act is not None and not isinstance(act, str) or act not in ACTS:
        raise ValueError(f"act must be one of {[a for a in ACTS if a]} or None")
    return ACTS[act]


def _linear_plan(bwd, x, weight, bias, res, pre, a, cf, ocf):
    """(C entry, device index, C shape, flags, workspace bytes, n, y's shape) of a call's checked tensors; res: the residual, or dy."""
    dev = _gpu(x)
    if weight.dim() != 2 or weight.dtype != x.dtype:
        raise ValueError("weight must be [n, k] of x's dtype")
    if weight.shape[1] > 1 and weight.stride(1) != 1:
        raise ValueError("the rows of weight must be contiguous")
    batch, rows, k, xs = _linear_layout(x, cf, cf or ocf, "x")
    n = weight.shape[0]
    if weight.shape[1] != k:
        raise ValueError(f"x has {k} channels, weight takes {weight.shape[1]}")
    if cf:
        shape = (batch, n) + tuple(x.shape[2:]) if ocf else (batch, rows, n)
    else:
        shape = (batch, n, rows) if ocf else tuple(x.shape[:-1]) + (n,)
    shape, rs = torch.Size(shape), (0, 0)
    if res is not None:
        name = "dy" if bwd else "residual"
        if res.shape != shape or res.dtype != x.dtype:
            raise ValueError(f"{name} must be {x.dtype} {list(shape)}")
        rs = _linear_layout(res, ocf, cf or ocf, name)[3]
    if bwd and a:
        if pre is None:
            raise ValueError("pre is required with an activation")
        if pre.shape != shape or pre.dtype != x.dtype or not pre.is_contiguous():
            raise ValueError(f"pre must be contiguous {x.dtype} {list(shape)}")
    _on_gpu(dev, weight=weight, bias=bias, residual=res, pre=pre)
    _f32((n,), bias=bias)
    flags = (LINEAR_X_MAPS if cf else 0) | (LINEAR_Y_MAPS if ocf else 0)
    s = _LinearShape(batch, rows, n, k, xs, rs, weight.stride(0))
    if bwd:
        need = _bytes("ssm2d_linear_bwd_workspace", x.dtype, s, a, flags)
    else:
        need = _bytes("ssm2d_linear_fwd_workspace", x.dtype, s, flags)
    return _entry("ssm2d_linear_bwd" if bwd else "ssm2d_linear_fwd", x.dtype), dev.index, s, flags, need, n, shape


def linear_fwd(x, weight, bias=None, residual=None, *, act=None, channels_first=False, out_channels_first=None, return_pre=False, y=None,
               stream=None):
    """y = act(x weight^T + bias) + residual. x: rows [..., k], or with
    ``channels_first`` maps [batch, k, ...] (the scan's layout); weight [n, k] of
    x's dtype, bias float32 [n]; act None, "relu", "silu" or "gelu" (by erf).
    ``out_channels_first`` (default: as x) lays y out the other way: from rows
    [batch, cells, k] to maps [batch, n, cells], or from maps to rows [batch,
    cells, n]. residual: y's shape and dtype. Returns y, or with ``return_pre``
    (y, pre): what act was applied to, for linear_bwd. ``y`` may be the residual."""
    a, cf = _act(act), bool(channels_first)
    ocf = cf if out_channels_first is None else bool(out_channels_first)
    key = ("linear", _meta(x), _meta(weight), _meta(bias), _meta(residual), a, cf, ocf)
    fn, index, s, flags, need, _, shape = _plans.get(key) or _keep(key, _linear_plan(False, x, weight, bias, residual, None, a, cf, ocf))
    dt = x.dtype
    y = _make("y", y, shape, dt, x, stream)
    pre = _make("pre", None, shape, dt, x, stream) if return_pre else None
    work = _workspace(need, x, stream)
    _launch(fn, index, stream, (x.data_ptr(), weight.data_ptr(), _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(pre), s, a, flags, _ptr(work), need))
    return (y, pre) if return_pre else y


def linear_bwd(x, weight, dy, pre=None, *, act=None, bias=True, channels_first=False, out_channels_first=None, out=None, stream=None):
    """Gradients of linear_fwd for dy, with the pre that it returned (needed with
    an activation): a dict dx, dweight (x's dtype) and, with ``bias``, dbias (float32
    [n]). The residual's gradient is dy. ``out`` may supply any of them."""
    a, cf = _act(act), bool(channels_first)
    ocf = cf if out_channels_first is None else bool(out_channels_first)
    if not a:
        pre = None
    key = ("linear_bwd", _meta(x), _meta(weight), _meta(dy), _meta(pre), a, cf, ocf)
    fn, index, s, flags, need, n, _ = _plans.get(key) or _keep(key, _linear_plan(True, x, weight, None, dy, pre, a, cf, ocf))
    out, dt = out or {}, x.dtype
    r = {"dx": _make("dx", out.get("dx"), x.shape, dt, x, stream), "dweight": _make("dweight", out.get("dweight"), weight.shape, dt, weight, stream)}
    if bias:
        r["dbias"] = _make("dbias", out.get("dbias"), (n,), torch.float32, x, stream)
    work = _workspace(need, x, stream)
    _launch(fn, index, stream, (x.data_ptr(), weight.data_ptr(), _ptr(pre), dy.data_ptr(), r["dx"].data_ptr(), r["dweight"].data_ptr(),
                                _ptr(r.get("dbias")), s, a, flags, _ptr(work), need))
    return r


# ------------------------------------------------------------------ block norm

def _rows_like(t, x, name, dtypes):
    """The row stride of an optional tensor of x's shape."""
    if t is None:
        return 0
    if t.shape != x.shape or t.dtype not in dtypes:
        raise ValueError(f"{name} must have x's shape, and {' or '.join(map(str, dtypes))}")
    return _norm_layout(t, False, name)[3]


def _norm_plan(bwd, x, weight, gate, residual, scale, next_weight, norm, groups, sigmoid, first, dout, dy):
    """(C entry, device index, C shape, flags, workspace bytes, n, dtype of out) of a call's checked tensors. dout: in the forward out's dtype."""
    dev = _gpu(x)
    rows, n, _, xs, _ = _norm_layout(x, False)
    if not 0 < groups or n % groups:
        raise ValueError("the channels must be a multiple of groups")
    if weight is not None and not norm:
        raise ValueError("weight belongs to the norm")
    _on_gpu(dev, weight=weight, gate=gate, residual=residual, scale=scale, next_weight=next_weight)
    _f32((n,), weight=weight, scale=scale, next_weight=next_weight)
    gs = _rows_like(gate, x, "gate", (x.dtype,))
    rs = _rows_like(residual, x, "residual", (x.dtype, torch.float32) if x.dtype != torch.float32 else (x.dtype,))
    os, ys = 0, 0
    rt = residual.dtype if residual is not None else None
    if bwd:
        if dy is not None and next_weight is None:
            raise ValueError("dy needs next_weight")
        if dout is None and dy is None:
            raise ValueError("dout or dy is required")
        rt = rt or (dout.dtype if dout is not None else x.dtype)
        if rt not in (x.dtype, torch.float32):
            raise ValueError("dout must have out's dtype")
        _on_gpu(dev, dout=dout, dy=dy)
        os, ys = _rows_like(dout, x, "dout", (rt,)), _rows_like(dy, x, "dy", (x.dtype,))
    else:
        rt = rt or dout or x.dtype
        if dout not in (None, rt) or rt not in (x.dtype, torch.float32):
            raise ValueError("out_dtype must be the residual's dtype, or x's or float32 without one")
    flags = ((NORM_ON if norm else 0) | (NORM_GATE_SIGMOID if sigmoid else 0) | (NORM_GATE_FIRST if first else 0)
             | (NORM_RESIDUAL_F32 if rt != x.dtype else 0))
    s = _NormShape(rows, n, groups, xs, gs, rs, os, ys)
    need = _bytes("ssm2d_block_norm_bwd_workspace", torch.float32, s, flags) if bwd else 0
    return _entry("ssm2d_block_norm_bwd" if bwd else "ssm2d_block_norm_fwd", x.dtype), dev.index, s, flags, need, n, rt


def _gate_act(act):
    if act not in ("silu", "sigmoid"):
        raise ValueError('gate_act must be "silu" or "sigmoid"')
    return act == "sigmoid"


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
    sig, norm, first, groups = _gate_act(gate_act), bool(norm), bool(gate_first), operator.index(groups)
    key = ("norm", _meta(x), _meta(weight), _meta(gate), _meta(residual), _meta(scale), _meta(next_weight), norm, groups, sig, first, out_dtype)
    fn, index, s, flags, _, _, rt = _plans.get(key) or _keep(key, _norm_plan(False, x, weight, gate, residual, scale, next_weight, norm, groups, sig,
                                                                           first, out_dtype, None))
    shape = x.shape
    out = _make("out", out, shape, rt, residual if residual is not None else x, stream)
    if next_weight is not None:
        y = _make("y", y, shape, x.dtype, x, stream)
    elif y is not None:
        raise ValueError("y needs next_weight")
    _launch(fn, index, stream, (x.data_ptr(), _ptr(gate), _ptr(residual), _ptr(weight), _ptr(scale), _ptr(next_weight), out.data_ptr(), _ptr(y), s,
                                float(eps), flags))
    return (out, y) if next_weight is not None else out


def block_norm_bwd(x, dout, dy=None, weight=None, *, gate=None, residual=None, scale=None, next_weight=None, norm=True, groups=1,
                   gate_act="silu", gate_first=False, eps=1e-5, out=None, stream=None):
    """Gradients of block_norm_fwd for dout (the gradient that reaches out
    otherwise than through y, of out's dtype; None: none) and, with next_weight,
    dy (None: none): a dict of dx and, of what was given, dgate, dresidual, and
    dweight, dscale, dnext_weight (float32 [n]). Nothing of the forward but its
    inputs is needed. ``out`` may supply any of them."""
    sig, norm, first, groups = _gate_act(gate_act), bool(norm), bool(gate_first), operator.index(groups)
    key = ("norm_bwd", _meta(x), _meta(weight), _meta(gate), _meta(residual), _meta(scale), _meta(next_weight), norm, groups, sig, first,
           _meta(dout), _meta(dy))
    fn, index, s, flags, need, n, rt = _plans.get(key) or _keep(key, _norm_plan(True, x, weight, gate, residual, scale, next_weight, norm, groups,
                                                                              sig, first, dout, dy))
    out, shape = out or {}, x.shape
    r = {"dx": _make("dx", out.get("dx"), shape, x.dtype, x, stream)}
    if gate is not None:
        r["dgate"] = _make("dgate", out.get("dgate"), shape, x.dtype, gate, stream)
    if residual is not None:
        r["dresidual"] = _make("dresidual", out.get("dresidual"), shape, rt, residual, stream)
    for name, t in (("dweight", weight), ("dscale", scale), ("dnext_weight", next_weight)):
        if t is not None:
            r[name] = _make(name, out.get(name), t.shape, torch.float32, t, stream)
    work = _workspace(need, x, stream)
    _launch(fn, index, stream, (x.data_ptr(), _ptr(gate), _ptr(residual), _ptr(weight), _ptr(scale), _ptr(next_weight), _ptr(dout), _ptr(dy),
                                r["dx"].data_ptr(), *(_ptr(r.get(k)) for k in ("dgate", "dresidual", "dweight", "dscale", "dnext_weight")), s,
                                float(eps), flags, _ptr(work), need))
    return r


# ------------------------------------------------------------------ recurrence

def _sequence_layout(t, maps, name):
    """(batch, tokens, channels, (batch stride, token or channel stride))"""
    if maps:
        b, c, tokens, sb, sc = _norm_layout(t, True, name)
        return b, tokens, c, (sb, sc)
    return _linear_layout(t, False, True, name)


def _gates(gates):
    if gates not in ("decay", "sigmoid"):
        raise ValueError('gates must be "decay" or "sigmoid"')
    return gates == "sigmoid"


def _recurrence_plan(bwd, x, g, sig, cu_seqlens, maps, rev, dh, states, step=False):
    """(C entry, device index, C shape, flags, workspace bytes, the states' shape) of a call's checked tensors."""
    dev = _gpu(x)
    if g.shape != x.shape or g.dtype != x.dtype:
        raise ValueError("g must match x in shape and dtype")
    if step:
        batch, channels = x.shape
        if channels > 1 and (x.stride(1) != 1 or g.stride(1) != 1):
            raise ValueError("the channels of x and g must be contiguous")
        tokens, xs, gs = 1, (x.stride(0), 0), (g.stride(0), 0)
    else:
        batch, tokens, channels, xs = _sequence_layout(x, maps, "x")
        gs = _sequence_layout(g, maps, "g")[3]
    ds, n_seq = (0, 0), 0
    if bwd:
        if dh.shape != x.shape or dh.dtype != x.dtype:
            raise ValueError("dh must match x in shape and dtype")
        ds = _sequence_layout(dh, maps, "dh")[3]
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous int32 [sequences + 1], at least one sequence")
        if batch != 1 or maps or rev:
            raise ValueError("packed sequences need batch 1, and go neither channels first nor in reverse")
        n_seq = cu_seqlens.numel() - 1
    shape = torch.Size((n_seq or batch, channels))
    _on_gpu(dev, g=g, cu_seqlens=cu_seqlens, dh=dh, **states)
    _f32(shape, **states)
    flags = (RECUR_SIGMOID if sig else 0) | (RECUR_MAPS if maps else 0) | (RECUR_REVERSE if rev else 0)
    s = _RecurrenceShape(batch, tokens, channels, n_seq, xs, gs, ds)
    need = _bytes("ssm2d_recurrence_bwd_workspace" if bwd else "ssm2d_recurrence_fwd_workspace", x.dtype, s, flags)
    return _entry("ssm2d_recurrence_bwd" if bwd else "ssm2d_recurrence_fwd", x.dtype), dev.index, s, flags, need, shape


def recurrence_fwd(x, g, *, gates="decay", h_init=None, cu_seqlens=None, channels_first=False, reverse=False, return_last_state=False, h=None,
                   h_last=None, stream=None):
    """h[t] = a[t] h[t - 1] + w[t] x[t] of each channel along the tokens: a =
    exp(g), w = 1 with ``gates`` "decay" (g the log decay), a = sigmoid(g), w = 1 - a
    with "sigmoid". x, g: [batch, tokens, channels], or with ``channels_first``
    [batch, channels, ...] with the cells as tokens; ``reverse`` goes from the last
    token to the first. Growing gates (g > 0) leave a state of 0 as it is; through
    tokens that another state passes their product has to be a float. With
    ``cu_seqlens`` (int32 [sequences + 1], batch 1) the tokens hold packed
    sequences; tokens behind the last one are left as they were. h_init: float32 [sequences, channels] or None (zeros). Returns h (x's
    shape and dtype), or (h, h_last)."""
    sig, maps, rev = _gates(gates), bool(channels_first), bool(reverse)
    key = ("recurrence", _meta(x), _meta(g), _meta(h_init), _meta(cu_seqlens), sig, maps, rev)
    fn, index, s, flags, need, states = _plans.get(key) or _keep(key, _recurrence_plan(False, x, g, sig, cu_seqlens, maps, rev, None,
                                                                                     {"h_init": h_init}))
    h = _make("h", h, x.shape, x.dtype, x, stream)
    if return_last_state or h_last is not None:
        h_last = _make("h_last", h_last, states, torch.float32, x, stream)
    work = _workspace(need, x, stream)
    _launch(fn, index, stream, (x.data_ptr(), g.data_ptr(), _ptr(h_init), _ptr(cu_seqlens), h.data_ptr(), _ptr(h_last), s, flags, _ptr(work), need))
    return (h, h_last) if return_last_state else h


def recurrence_bwd(x, g, dh, *, gates="decay", h_init=None, dh_last=None, cu_seqlens=None, channels_first=False, reverse=False, out=None,
                   stream=None):
    """Gradients of recurrence_fwd for dh = dL/dh and dh_last = dL/dh_last (None:
    zeros): a dict dx, dg (x's dtype), and dh_init (float32) when h_init or
    dh_last is given or ``out`` holds it. ``out`` may supply any of them."""
    sig, maps, rev = _gates(gates), bool(channels_first), bool(reverse)
    key = ("recurrence_bwd", _meta(x), _meta(g), _meta(h_init), _meta(dh_last), _meta(cu_seqlens), _meta(dh), sig, maps, rev)
    fn, index, s, flags, need, states = _plans.get(key) or _keep(key, _recurrence_plan(True, x, g, sig, cu_seqlens, maps, rev, dh,
                                                                                     {"h_init": h_init, "dh_last": dh_last}))
    out = out or {}
    r = {n: _make(n, out.get(n), x.shape, x.dtype, x, stream) for n in ("dx", "dg")}
    if h_init is not None or dh_last is not None or out.get("dh_init") is not None:
        r["dh_init"] = _make("dh_init", out.get("dh_init"), states, torch.float32, x, stream)
    work = _workspace(need, x, stream)
    _launch(fn, index, stream, (x.data_ptr(), g.data_ptr(), _ptr(h_init), _ptr(cu_seqlens), dh.data_ptr(), _ptr(dh_last), r["dx"].data_ptr(),
                                r["dg"].data_ptr(), _ptr(r.get("dh_init")), s, flags, _ptr(work), need))
    return r


def recurrence_step(x, g, state, *, gates="decay", h=None, stream=None):
    """One token of the recurrence for each batch entry: x, g [batch, channels];
    state: float32 [batch, channels], updated in place. Returns h (x's shape and
    dtype)."""
    if x.dim() != 2:
        raise ValueError("x and g must be [batch, channels]")
    if state is None:
        raise ValueError("state is required")
    sig = _gates(gates)
    key = ("step", _meta(x), _meta(g), _meta(state), sig)
    fn, index, s, flags, need, _ = _plans.get(key) or _keep(key, _recurrence_plan(False, x, g, sig, None, False, False, None, {"state": state}, True))
    h = _make("h", h, x.shape, x.dtype, x, stream)
    at = state.data_ptr()
    _launch(fn, index, stream, (x.data_ptr(), g.data_ptr(), at, None, h.data_ptr(), at, s, flags, None, need))
    return h
