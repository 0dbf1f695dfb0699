"""Python binding of the operators around the 2D scan (include/ssm2d_ops.h):
layer norm, rotary positions with several axes, and the gated delta rule.

Like the scan's binding it only checks tensors and passes pointers, strides and
the HIP stream to libssm2d.so; every operator runs in the library's kernels.

    y = layer_norm_fwd(x, weight, bias)                 # rows, or channels_first=True maps
    g = layer_norm_bwd(x, weight, mean, rstd, dy)       # dict: dx, dweight, dbias
    q, k = rope_fwd(q, k, positions, inv_freq, sections)
    o = gated_delta_fwd(q, k, v, g, beta)               # sequences, packed with cu_seqlens=...
    g = gated_delta_bwd(q, k, v, g, beta, do)           # dict: dq, dk, dv, dg, dbeta, dh_init
    o = gated_delta_step(q, k, v, g, beta, state)       # one token, state updated in place

x, q, k, v and gradients of them: float32 or bfloat16; weights, statistics, g,
beta and states: float32. Inputs may be strided views (inner dim contiguous);
outputs are dense, and take no part in autograd: gradients come from the _bwd
entries (examples/map_mixer.py wraps them). Without ``stream`` a call runs on the current stream of its
tensors' device; with one, its outputs are allocated on that stream too, and
ordering the inputs' producers before it is the caller's.
"""
from __future__ import annotations

import ctypes
import functools
import operator

import torch

from . import ERR_HIP, OK, Ssm2dError, load_library

__all__ = ["layer_norm_fwd", "layer_norm_bwd", "rope_fwd", "rope_bwd", "gated_delta_fwd", "gated_delta_bwd", "gated_delta_step"]

LN_MAX_N, ROPE_MAX_AXES, ROPE_MAX_D, DELTA_MAX_DK, DELTA_MAX_DV = 16384, 4, 1024, 128, 1024
ROPE_INTERLEAVED, ROPE_INVERSE = 1, 2

_vp, _i64 = ctypes.c_void_p, ctypes.c_int64


class _RopeShape(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64), ("heads_q", _i64), ("heads_k", _i64), ("d", _i64), ("q_stride", _i64 * 3),
                ("k_stride", _i64 * 3), ("n_axes", _i64), ("sections", _i64 * ROPE_MAX_AXES), ("pos_stride", _i64 * 2)]


class _DeltaShape(ctypes.Structure):
    _fields_ = [("batch", _i64), ("tokens", _i64), ("n_seq", _i64), ("heads_qk", _i64), ("heads", _i64), ("d_k", _i64), ("d_v", _i64),
                ("q_stride", _i64 * 3), ("k_stride", _i64 * 3), ("v_stride", _i64 * 3), ("do_stride", _i64 * 3), ("g_stride", _i64 * 3),
                ("beta_stride", _i64 * 3)]


_SIGNATURES = {
    "ssm2d_layer_norm_fwd": [_vp] * 6 + [_i64] * 5 + [ctypes.c_float, _vp],
    "ssm2d_layer_norm_bwd": [_vp] * 8 + [_i64] * 7 + [_vp],
    "ssm2d_rope": [_vp] * 6 + [ctypes.POINTER(_RopeShape), ctypes.c_uint32, _vp],
    "ssm2d_gated_delta_fwd": [_vp] * 9 + [ctypes.POINTER(_DeltaShape), ctypes.c_float, _vp],
    "ssm2d_gated_delta_bwd": [_vp] * 15 + [ctypes.POINTER(_DeltaShape), ctypes.c_float, _vp],
    "ssm2d_gated_delta_step": [_vp] * 7 + [ctypes.POINTER(_DeltaShape), ctypes.c_float, _vp],
}
_bound = {}


def _entry(name, dtype):
    """The C entry ``name`` for tensors of ``dtype`` (its _bf16 variant)."""
    f = _bound.get((name, dtype))
    if f is None:
        if dtype not in (torch.float32, torch.bfloat16):
            raise TypeError("tensors must be float32 or bfloat16")
        f = getattr(load_library(), name if dtype == torch.float32 else name + "_bf16")
        f.argtypes, f.restype = _SIGNATURES[name], ctypes.c_int
        _bound[name, dtype] = f
    return f


# The current stream's handle: 0.1 us where torch offers it as an integer, 2 us through a Stream object.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _run(fn, dev, stream, args):
    """Calls fn(*args, stream) with ``dev`` current; a status becomes an exception."""
    handle = stream.cuda_stream if stream is not None else _raw_stream(dev.index)
    if dev.index == torch.cuda.current_device():
        s = fn(*args, handle)
    else:
        with torch.cuda.device(dev):
            s = fn(*args, handle)
    if s != OK:
        raise Ssm2dError(s, fn.__name__ + (f" ({load_library().ssm2d_last_hip_error().decode()})" if s == ERR_HIP else ""))


def _new(shape, dtype, dev, stream):
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def _ptr(t):
    return t.data_ptr() if t is not None else None


def _on_gpu(dev, **tensors):
    if dev.type != "cuda":
        raise ValueError("tensors must be on a GPU")
    for name, t in tensors.items():
        if t is not None and t.device != dev:
            raise ValueError(f"{name} must be on the same device as the other tensors")


def _f32(shape, **tensors):
    """Optional dense float32 tensors of one shape."""
    for name, t in tensors.items():
        if t is not None and (t.dtype != torch.float32 or t.shape != shape or not t.is_contiguous()):
            raise ValueError(f"{name} must be contiguous float32 {list(shape)}")


def _like(name, t, ref, stream):
    """An output like a tensor of the call: given, or allocated."""
    if t is None and stream is None and ref.is_contiguous():
        return torch.empty_like(ref)
    return _out(name, t, ref.shape, ref.dtype, ref.device, stream)


def _out(name, t, shape, dtype, dev, stream):
    if t is None:
        return _new(shape, dtype, dev, stream)
    if t.shape != shape or t.dtype != dtype or t.device != dev or not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous {dtype} {list(shape)} on the inputs' device")
    return t


# ------------------------------------------------------------------ layer norm

def _norm_layout(x, channels_first, name="x"):
    """(batch, n, cells, batch stride, channel stride) of rows [..., n] or maps [batch, n, ...]."""
    if channels_first:
        if x.dim() < 2:
            raise ValueError(f"{name} must be [batch, channels, ...]")
        if 0 in x.shape[2:]:
            return x.shape[0], x.shape[1], 0, x.stride(0), x.stride(1)
        cells = 1
        for size, stride in zip(reversed(x.shape[2:]), reversed(x.stride()[2:])):
            if size != 1 and stride != cells:
                raise ValueError(f"the cells of {name} must be contiguous")
            cells *= size
        return x.shape[0], x.shape[1], cells, x.stride(0), x.stride(1)
    if x.dim() < 1:
        raise ValueError(f"{name} must be [..., channels]")
    n = x.shape[-1]
    if n == 0:
        return x.shape[:-1].numel(), 0, 1, 0, 1
    if x.dim() != 2:
        try:
            x = x.view(-1, n)
        except RuntimeError:
            raise ValueError(f"the rows of {name} must lie at one stride") from None
    if n > 1 and x.shape[0] and x.stride(1) != 1:
        raise ValueError(f"the channels of {name} must be contiguous")
    return x.shape[0], n, 1, x.stride(0), 1


def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, *, channels_first=False, return_stats=False, y=None, stream=None):
    """Layer norm over the last dim of x, or over dim 1 of maps [batch,
    channels, ...] with ``channels_first`` (the scan's layout). weight, bias:
    float32 [channels] or None. Returns y (x's dtype), or (y, mean, rstd) with
    ``return_stats``: float32, of x's shape without the channels."""
    fn, dev = _entry("ssm2d_layer_norm_fwd", x.dtype), x.device
    batch, n, cells, sb, sn = _norm_layout(x, channels_first)
    _on_gpu(dev, weight=weight, bias=bias)
    _f32((n,), weight=weight, bias=bias)
    y = _like("y", y, x, stream)
    mean = rstd = None
    if return_stats:
        shape = x.shape[:1] + x.shape[2:] if channels_first else x.shape[:-1]
        mean, rstd = _new(shape, torch.float32, dev, stream), _new(shape, torch.float32, dev, stream)
    _run(fn, dev, stream, (x.data_ptr(), _ptr(weight), _ptr(bias), y.data_ptr(), _ptr(mean), _ptr(rstd), batch, n, cells, sb, sn,
                           float(eps)))
    return (y, mean, rstd) if return_stats else y


def layer_norm_bwd(x, weight, mean, rstd, dy, *, channels_first=False, out=None, stream=None):
    """Gradients of layer_norm_fwd for dy, with the forward's mean and rstd: a
    dict dx (x's dtype), dweight, dbias (float32 [channels]). ``out`` may supply
    any of them."""
    fn, dev = _entry("ssm2d_layer_norm_bwd", x.dtype), x.device
    batch, n, cells, sb, sn = _norm_layout(x, channels_first)
    if dy.shape != x.shape or dy.dtype != x.dtype:
        raise ValueError("dy must match x in shape and dtype")
    if mean is None or rstd is None:
        raise ValueError("mean and rstd are required")
    _, _, _, gb, gn = _norm_layout(dy, channels_first, "dy")
    _on_gpu(dev, weight=weight, mean=mean, rstd=rstd, dy=dy)
    _f32((n,), weight=weight)
    _f32(x.shape[:1] + x.shape[2:] if channels_first else x.shape[:-1], mean=mean, rstd=rstd)
    out = out or {}
    r = {"dx": _like("dx", out.get("dx"), x, stream)}
    for name in ("dweight", "dbias"):
        r[name] = (_out(name, out.get(name), (n,), torch.float32, dev, stream) if weight is None
                   else _like(name, out.get(name), weight, stream))
    _run(fn, dev, stream, (x.data_ptr(), _ptr(weight), mean.data_ptr(), rstd.data_ptr(), dy.data_ptr(), r["dx"].data_ptr(),
                           r["dweight"].data_ptr(), r["dbias"].data_ptr(), batch, n, cells, sb, sn, gb, gn))
    return r


# ------------------------------------------------------------------ rotary positions

@functools.lru_cache(maxsize=256)
def _rope_shape(batch, tokens, hq, hk, d, qs, ks, sections, pos):
    return _RopeShape(batch, tokens, hq, hk, d, qs, ks, len(sections), sections + (0,) * (ROPE_MAX_AXES - len(sections)), pos)


def _sections(sections):
    """(the sections as integers, the pairs they make)."""
    if not 1 <= len(sections) <= ROPE_MAX_AXES:
        raise ValueError(f"1 to {ROPE_MAX_AXES} sections")
    sections = tuple(map(operator.index, sections))
    return sections, sum(sections)


def _strides(t, name):
    if t.shape[3] > 1 and t.stride(3) != 1:
        raise ValueError(f"the last dim of {name} must be contiguous")
    return t.stride()[:3]


def _rope(q, k, positions, inv_freq, sections, interleaved, inverse, q_out, k_out, stream):
    fn, dev = _entry("ssm2d_rope", q.dtype), q.device
    if q.dim() != 4:
        raise ValueError("q must be [batch, tokens, heads, d]")
    B, T, hq, d = q.shape
    sections, pairs = _sections(tuple(sections))
    axes = len(sections)
    if positions.dtype != torch.int32 or positions.shape not in ((axes, T), (axes, B, T)):
        raise ValueError("positions must be int32 [axes, tokens] or [axes, batch, tokens]")
    ps = positions.stride()
    if T > 1 and ps[-1] != 1:
        raise ValueError("the last dim of positions must be contiguous")
    if inv_freq.dtype != torch.float32 or inv_freq.shape != (pairs,) or not inv_freq.is_contiguous():
        raise ValueError(f"inv_freq must be contiguous float32 [{pairs}]")
    qs, ks, hk, kp, kop = q.stride(), (0, 0, 0), 0, None, None
    if d > 1 and qs[3] != 1:
        raise ValueError("the last dim of q must be contiguous")
    if k is not None:
        if k.dim() != 4 or k.dtype != q.dtype or k.shape[:2] != (B, T) or k.shape[3] != d:
            raise ValueError("k must be [batch, tokens, heads, d] like q, but for the heads")
        hk, ks = k.shape[2], _strides(k, "k")
        k_out = _like("k_out", k_out, k, stream)
        if hk:
            kp, kop = k.data_ptr(), k_out.data_ptr()
    _on_gpu(dev, k=k, positions=positions, inv_freq=inv_freq)
    q_out = _like("q_out", q_out, q, stream)
    shape = _rope_shape(B, T, hq, hk, d, qs[:3], ks, sections, (ps[0], ps[1] if len(ps) == 3 else 0))
    _run(fn, dev, stream, (q.data_ptr(), kp, positions.data_ptr(), inv_freq.data_ptr(), q_out.data_ptr(), kop, shape,
                           (ROPE_INTERLEAVED if interleaved else 0) | (ROPE_INVERSE if inverse else 0)))
    return q_out, (k_out if k is not None else None)


def rope_fwd(q, k, positions, inv_freq, sections, *, interleaved=False, q_out=None, k_out=None, stream=None):
    """Turns the pairs of q [batch, tokens, heads, d] and k (its own number of
    heads, or None) by positions[axis of the pair] * inv_freq[pair]. sections:
    pairs of each axis, e.g. (rows, columns) of a map or (time, height, width)
    of a clip; positions: int32 [axes, tokens] or [axes, batch, tokens];
    inv_freq: float32 [pairs]. Pair p is dims (p, pairs + p), or (2p, 2p + 1)
    when ``interleaved``; dims past the pairs are copied. Returns (q, k)."""
    return _rope(q, k, positions, inv_freq, sections, interleaved, False, q_out, k_out, stream)


def rope_bwd(dq, dk, positions, inv_freq, sections, *, interleaved=False, q_out=None, k_out=None, stream=None):
    """Gradients of rope_fwd with respect to its q and k, for those of its
    outputs: the turn by the opposite angles. Returns (dq, dk)."""
    return _rope(dq, dk, positions, inv_freq, sections, interleaved, True, q_out, k_out, stream)


# ------------------------------------------------------------------ gated delta rule

@functools.lru_cache(maxsize=256)
def _delta_shape(batch, tokens, n_seq, hk, h, dk, dv, qs, ks, vs, os, gs, bs):
    return _DeltaShape(batch, tokens, n_seq, hk, h, dk, dv, qs, ks, vs, os, gs, bs)


def _scale(scale, d_k):
    return max(d_k, 1) ** -0.5 if scale is None else float(scale)


def _delta_check(q, k, v, g, beta, cu_seqlens, do=None):
    """(device, sequences, the C shape) of one call's checked tensors [batch, tokens, heads, d]."""
    if q.dim() != 4 or k.shape != q.shape or v.dim() != 4 or v.shape[:2] != q.shape[:2]:
        raise ValueError("q and k must be [batch, tokens, heads_qk, d_k], v [batch, tokens, heads, d_v]")
    B, T, hk, dk = q.shape
    h, dv = v.shape[2:]
    if (h % hk if hk else h) != 0:
        raise ValueError("heads must be a multiple of heads_qk")
    if k.dtype != q.dtype or v.dtype != q.dtype:
        raise TypeError("q, k and v must have one dtype")
    for name, t in (("g", g), ("beta", beta)):
        if t.dtype != torch.float32 or t.shape != (B, T, h):
            raise ValueError(f"{name} must be float32 [batch, tokens, heads]")
    n_seq = 0
    if cu_seqlens is not None:
        if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or cu_seqlens.numel() < 2 or not cu_seqlens.is_contiguous():
            raise ValueError("cu_seqlens must be contiguous int32 [sequences + 1], at least one sequence")
        if B != 1:
            raise ValueError("packed sequences need batch 1")
        n_seq = cu_seqlens.numel() - 1
    os = (0, 0, 0)
    if do is not None:
        if do.shape != v.shape or do.dtype != v.dtype:
            raise ValueError("do must match v in shape and dtype")
        os = _strides(do, "do")
    _on_gpu(q.device, k=k, v=v, g=g, beta=beta, cu_seqlens=cu_seqlens, do=do)
    return q.device, n_seq or B, _delta_shape(B, T, n_seq, hk, h, dk, dv, _strides(q, "q"), _strides(k, "k"), _strides(v, "v"), os,
                                              g.stride(), beta.stride())


def gated_delta_fwd(q, k, v, g, beta, *, scale=None, h_init=None, cu_seqlens=None, return_last_state=False, o=None, h_last=None,
                    stream=None):
    """The gated delta rule over sequences: per head a state S [d_k, d_v],
    S' = exp(g) S, u = beta (v - S'^T k), S = S' + k u^T, o = scale S^T q.
    q, k: [batch, tokens, heads_qk, d_k]; v: [batch, tokens, heads, d_v] (heads a
    multiple of heads_qk); g, beta: float32 [batch, tokens, heads]. ``scale``
    defaults to d_k ** -0.5. With ``cu_seqlens`` (int32 [sequences + 1]) the one
    batch entry holds packed sequences. h_init: float32 [sequences, heads, d_k,
    d_v] or None (zeros). Returns o (v's shape and dtype), or (o, h_last)."""
    fn = _entry("ssm2d_gated_delta_fwd", q.dtype)
    dev, seqs, shape = _delta_check(q, k, v, g, beta, cu_seqlens)
    states = (seqs, v.shape[2], q.shape[3], v.shape[3])
    _on_gpu(dev, h_init=h_init)
    _f32(states, h_init=h_init)
    o = _like("o", o, v, stream)
    if return_last_state or h_last is not None:
        h_last = _out("h_last", h_last, states, torch.float32, dev, stream)
    _run(fn, dev, stream, (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(h_init), _ptr(cu_seqlens),
                           o.data_ptr(), _ptr(h_last), shape, _scale(scale, q.shape[3])))
    return (o, h_last) if return_last_state else o


def gated_delta_bwd(q, k, v, g, beta, do, *, scale=None, h_init=None, dh_last=None, cu_seqlens=None, out=None, stream=None):
    """Gradients of gated_delta_fwd for do = dL/do and dh_last = dL/dh_last
    (None: zeros): a dict dq, dk, dv (their inputs' dtype), dg, dbeta (float32),
    and dh_init when h_init or dh_last is given or ``out`` holds it. ``out`` may supply any of them."""
    fn = _entry("ssm2d_gated_delta_bwd", q.dtype)
    dev, seqs, shape = _delta_check(q, k, v, g, beta, cu_seqlens, do)
    states = (seqs, v.shape[2], q.shape[3], v.shape[3])
    _on_gpu(dev, h_init=h_init, dh_last=dh_last)
    _f32(states, h_init=h_init, dh_last=dh_last)
    out = out or {}
    r = {n: _like(n, out.get(n), t, stream) for n, t in (("dq", q), ("dk", k), ("dv", v), ("dg", g), ("dbeta", beta))}
    if h_init is not None or dh_last is not None or out.get("dh_init") is not None:
        r["dh_init"] = _out("dh_init", out.get("dh_init"), states, torch.float32, dev, stream)
    _run(fn, dev, stream, (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), _ptr(h_init), _ptr(cu_seqlens),
                           do.data_ptr(), _ptr(dh_last), *(r[n].data_ptr() for n in ("dq", "dk", "dv", "dg", "dbeta")), _ptr(r.get("dh_init")),
                           shape, _scale(scale, q.shape[3])))
    return r


def gated_delta_step(q, k, v, g, beta, state, *, scale=None, o=None, stream=None):
    """One token of the gated delta rule for each batch entry: q, k [batch,
    heads_qk, d_k], v [batch, heads, d_v], g, beta [batch, heads]; or a few
    tokens, all with a token dim after the batch. state: float32 [batch, heads,
    d_k, d_v], updated in place. Returns o (v's shape and dtype)."""
    fn = _entry("ssm2d_gated_delta_step", q.dtype)
    if state is None:
        raise ValueError("state is required")
    if q.dim() == 3:  # one token: as [batch, 1, heads, d] without making the views
        (B, hk, dk), (_, h, dv) = q.shape, v.shape if v.dim() == 3 else (0, 0, 0)
        dev = q.device
        if k.shape != q.shape or v.shape != (B, h, dv) or g.shape != (B, h) or beta.shape != (B, h) or (h % hk if hk else h) != 0:
            raise ValueError("one token: q and k [batch, heads_qk, d_k], v [batch, heads, d_v], g and beta [batch, heads]")
        if k.dtype != q.dtype or v.dtype != q.dtype:
            raise TypeError("q, k and v must have one dtype")
        if g.dtype != torch.float32 or beta.dtype != torch.float32:
            raise ValueError("g and beta must be float32")
        qs, ks, vs, gs, bs = q.stride(), k.stride(), v.stride(), g.stride(), beta.stride()
        if (dk > 1 and (qs[2] != 1 or ks[2] != 1)) or (dv > 1 and vs[2] != 1):
            raise ValueError("the last dims of q, k and v must be contiguous")
        _on_gpu(dev, k=k, v=v, g=g, beta=beta, state=state)
        shape = _delta_shape(B, 1, 0, hk, h, dk, dv, (qs[0], 0, qs[1]), (ks[0], 0, ks[1]), (vs[0], 0, vs[1]), (0, 0, 0),
                             (gs[0], 0, gs[1]), (bs[0], 0, bs[1]))
    else:
        dev, B, shape = _delta_check(q, k, v, g, beta, None)
        h, dk, dv = v.shape[2], q.shape[3], v.shape[3]
        _on_gpu(dev, state=state)
    _f32((B, h, dk, dv), state=state)
    o = _like("o", o, v, stream)
    _run(fn, dev, stream, (q.data_ptr(), k.data_ptr(), v.data_ptr(), g.data_ptr(), beta.data_ptr(), state.data_ptr(), o.data_ptr(),
                           shape, _scale(scale, dk)))
    return o
