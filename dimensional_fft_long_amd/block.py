"""The residual block around the gated convolution: argument marshalling for the
norm, join, dropout and gated feed-forward entry points of
``include/hyenand.h`` (formulas there).

Tensors are [B, C, *dims] with one to three grid axes, contiguous, float32 or
bfloat16; per-channel parameters are float32 [C].  A layer::

    h = block_norm(x, w1)
    m = gated_fftconv(h, alpha, beta, K)
    x, h = block_join(x, m, gate=g, scale=s, w_post=w2, w_pre=w3, p=0.1, rng=rng)
    x, h = block_join(x, gated_ffn(h, Wg, Wu, Wd), scale=s2, w_pre=w4)

``rng`` is an int64 device tensor [seed, offset]; masks are functions of it and
of the element's index alone, and are drawn again in the backward.  Give every
use other words: advance the offset by ceil(numel / 4), out of place between
forward and backward.

Every call runs on ``stream`` (default: the current stream of the tensors'
device).  Calls without a ``workspace`` take one from the package's cache, or,
while the stream is being captured, one of the graph's own memory.
"""
from __future__ import annotations

import ctypes
import functools
import threading

import torch
from torch.autograd.function import once_differentiable

from . import (OK, HyenandError, _check_out, _dims_arr, _dtype_code, _ws_bytes, _ws_cache, get_lib)

ACTS = {"none": 0, "sigmoid": 1, "silu": 2, "gelu": 3}

_P = ctypes.c_void_p


class _Join(ctypes.Structure):
    """hyenand_join."""
    _fields_ = [(k, _P) for k in ("gate", "scale", "w_post", "w_pre", "rng")] + \
               [("p", ctypes.c_double), ("eps", ctypes.c_float), ("gate_act", ctypes.c_int)]


class _JoinGrads(ctypes.Structure):
    """hyenand_join_grads."""
    _fields_ = [(k, _P) for k in ("dx", "dm", "dgate", "dscale", "dw_post", "dw_pre")]


def _declare(lib) -> None:
    P, I, SZ, F, D = ctypes.c_void_p, ctypes.c_int, ctypes.c_size_t, ctypes.c_float, ctypes.c_double
    J, G = ctypes.POINTER(_Join), ctypes.POINTER(_JoinGrads)
    for name, res, args in (
            ("hyenand_block_norm_fwd", I, [P, P, P, I, I, I, P, I, F, P]),
            ("hyenand_block_norm_bwd_workspace_bytes", SZ, [I, I, I, P, I]),
            ("hyenand_block_norm_bwd", I, [P, P, P, P, P, I, I, I, P, I, F, P, SZ, P]),
            ("hyenand_block_join_fwd", I, [P, P, J, P, P, I, I, I, P, I, P]),
            ("hyenand_block_join_bwd_workspace_bytes", SZ, [I, I, I, P, I]),
            ("hyenand_block_join_bwd", I, [P, P, J, P, P, G, I, I, I, P, I, P, SZ, P]),
            ("hyenand_dropout", I, [P, P, ctypes.c_int64, I, D, P, P]),
            ("hyenand_gated_ffn_workspace_bytes", SZ, [I, I, I, I, P, I]),
            ("hyenand_gated_ffn_bwd_workspace_bytes", SZ, [I, I, I, I, P, I]),
            ("hyenand_gated_ffn_fwd", I, [P, P, P, P, P, I, I, I, I, P, I, I, P, SZ, P]),
            ("hyenand_gated_ffn_bwd", I, [P] * 9 + [I, I, I, I, P, I, I, P, SZ, P])):
        f = getattr(lib, name)
        f.restype, f.argtypes = res, args


# ------------------------------------------------------------------- helpers

def _x(t, name="x"):
    if not isinstance(t, torch.Tensor) or not t.is_cuda or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous device tensor")
    if not 3 <= t.dim() <= 5:
        raise ValueError(f"{name} must be [B, C, *dims] with one to three grid axes, got {tuple(t.shape)}")
    return _dtype_code(t.dtype)


def _like(t, name, x, optional=False):
    if t is None and optional:
        return
    if not isinstance(t, torch.Tensor) or t.dtype is not x.dtype or t.device != x.device or not t.is_contiguous():
        raise TypeError(f"{name} must be a contiguous {x.dtype} tensor on {x.device}")
    if t.shape != x.shape:
        raise ValueError(f"{name} must have the shape {tuple(x.shape)}, got {tuple(t.shape)}")


def _channel(t, name, x, optional=False):
    if t is None and optional:
        return
    if not isinstance(t, torch.Tensor) or t.dtype is not torch.float32 or t.device != x.device or \
            not t.is_contiguous() or t.dim() != 1 or t.shape[0] != x.shape[1]:
        raise TypeError(f"{name} must be a contiguous float32 tensor of {x.shape[1]} elements on {x.device}")


def _rng(rng, p, device):
    p = float(p)
    if not 0.0 <= p < 1.0:
        raise ValueError(f"p must be in [0, 1), got {p}")
    if p > 0.0 and (not isinstance(rng, torch.Tensor) or rng.dtype != torch.int64 or tuple(rng.shape) != (2,) or
                    rng.device != device or not rng.is_contiguous()):
        raise TypeError(f"rng must be an int64 tensor [seed, offset] on {device}")
    return p


def _act(name, allowed):
    if name not in allowed:
        raise ValueError(f"activation must be one of {', '.join(allowed)}, got {name!r}")
    return ACTS[name]


def _ptr(t):
    return None if t is None else t.data_ptr()


@functools.lru_cache(maxsize=1024)
def _shape(shape):
    """(B, C, d, extents) of a tensor's shape, as the entry points take them."""
    dims = tuple(int(v) for v in shape[2:])
    return int(shape[0]), int(shape[1]), len(dims), _dims_arr(dims)


# The current stream's handle; the public call builds a Stream object for it,
# which costs as much as a small kernel.
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or \
    (lambda index: torch.cuda.current_stream(index).cuda_stream)


def _call(device, stream, inputs, body):
    """body(stream handle) with the tensors' device and the call's stream
    current, so that outputs and workspaces come from that stream's memory;
    inputs of another stream are marked as used on it."""
    if stream is None and device.index == torch.cuda.current_device():
        return body(_raw_stream(device.index))
    with torch.cuda.device(device):
        if stream is None:
            return body(_raw_stream(device.index))
        if stream.device != device:
            raise ValueError(f"the stream must be one of {device}, got {stream.device}")
        foreign = stream != torch.cuda.current_stream(device)
        with torch.cuda.stream(stream):
            r = body(stream.cuda_stream)
            if foreign and not torch.cuda.is_current_stream_capturing():
                for t in inputs:
                    if t is not None and t.numel():
                        t.record_stream(stream)
    return r


def _ws(workspace, kind, nbytes, device, st):
    """(buffer, bytes): the caller's workspace, or one of the cache, one per kind,
    device, stream and host thread (the launches of two threads' calls may
    interleave on one stream), as large as its largest call.  A captured call
    takes memory of its graph instead: a cached buffer would be shared with other
    graphs and with eager calls, which a replay does not wait for."""
    if workspace is not None:
        return workspace, _ws_bytes(workspace, device)
    if torch.cuda.is_current_stream_capturing():
        return torch.empty(max(nbytes, 8), dtype=torch.uint8, device=device), nbytes
    key = (kind, device.index, st, threading.get_ident())
    buf = _ws_cache.get(key)
    if buf is None or buf.numel() < nbytes:
        _ws_cache.pop(key, None)
        buf = None  # freed, in its stream's order, before the larger one is asked for
        buf = _ws_cache[key] = torch.empty(max(nbytes, 8), dtype=torch.uint8, device=device)
    return buf, nbytes


def _done(rc, what):
    if rc != OK:
        raise HyenandError(rc, what)


def _out(t, name, like, inputs):
    """A caller's output (or a new one): shape and dtype of ``like``, apart from every input."""
    if t is None:
        return torch.empty_like(like)
    _check_out(t, name, like.shape, like.dtype, like.device)
    a0 = t.data_ptr()
    a1 = a0 + t.numel() * t.element_size()
    for i in inputs:
        if i is not None and a0 < i.data_ptr() + i.numel() * i.element_size() and i.data_ptr() < a1:
            raise ValueError(f"{name} must not overlap the inputs or another output")
    return t


# ---------------------------------------------------------------------- norm

def block_norm_fwd(x, w, eps: float = 1e-6, h=None, stream=None):
    """h = x r w, r the reciprocal root mean square of x over its channels."""
    dt = _x(x)
    _channel(w, "w", x)

    def body(st):
        o = _out(h, "h", x, (x, w))
        _done(get_lib().hyenand_block_norm_fwd(x.data_ptr(), w.data_ptr(), o.data_ptr(), *_shape(x.shape), dt, eps, st),
              "block_norm_fwd")
        return o

    return _call(x.device, stream, (x, w), body)


def block_norm_bwd(x, w, dh, eps: float = 1e-6, workspace=None, stream=None):
    """(dx, dw) of block_norm_fwd for the gradient dh of h."""
    dt = _x(x)
    _channel(w, "w", x)
    _like(dh, "dh", x)

    def body(st):
        lib, shape = get_lib(), _shape(x.shape)
        dx, dw = torch.empty_like(x), torch.empty_like(w)
        ws, nb = _ws(workspace, "block_norm_bwd", lib.hyenand_block_norm_bwd_workspace_bytes(*shape, dt), x.device, st)
        _done(lib.hyenand_block_norm_bwd(x.data_ptr(), w.data_ptr(), dh.data_ptr(), dx.data_ptr(), dw.data_ptr(),
                                         *shape, dt, eps, ws.data_ptr(), nb, st), "block_norm_bwd")
        return dx, dw

    return _call(x.device, stream, (x, w, dh), body)


class BlockNormFunction(torch.autograd.Function):
    """block_norm_fwd and its backward as one differentiable operation."""

    @staticmethod
    def forward(ctx, x, w, eps):
        ctx.save_for_backward(x, w)
        ctx.eps = eps
        return block_norm_fwd(x, w, eps)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, w = ctx.saved_tensors
        dx, dw = block_norm_bwd(x, w, dh.contiguous(), ctx.eps)
        return dx, dw, None


def block_norm(x, w, eps: float = 1e-6):
    """Differentiable norm over the channels (BlockNormFunction)."""
    return BlockNormFunction.apply(x, w, eps)


# ---------------------------------------------------------------------- join

def _join(x, m, gate, scale, w_post, w_pre, gate_act, eps, p, rng):
    dt = _x(x)
    _like(m, "m", x)
    _like(gate, "gate", x, optional=True)
    for t, nm in ((scale, "scale"), (w_post, "w_post"), (w_pre, "w_pre")):
        _channel(t, nm, x, optional=True)
    p = _rng(rng, p, x.device)
    act = _act(gate_act, ("none", "sigmoid", "silu"))
    return dt, _Join(_ptr(gate), _ptr(scale), _ptr(w_post), _ptr(w_pre), _ptr(rng) if p else None, p, eps, act)


def block_join_fwd(x, m, gate=None, scale=None, w_post=None, w_pre=None, gate_act: str = "sigmoid", eps: float = 1e-6,
                   p: float = 0.0, rng=None, out=None, h=None, stream=None):
    """(out, h): out = x + dropout(scale * gate_act(gate) * norm(m; w_post)) and
    h = norm(out; w_pre), h None where w_pre is."""
    dt, j = _join(x, m, gate, scale, w_post, w_pre, gate_act, eps, p, rng)
    ins = (x, m, gate, scale, w_post, w_pre)
    if w_pre is None and h is not None:
        raise ValueError("h is computed only with w_pre")

    def body(st):
        o = _out(out, "out", x, ins)
        hh = None if w_pre is None else _out(h, "h", x, ins + (o,))
        _done(get_lib().hyenand_block_join_fwd(x.data_ptr(), m.data_ptr(), ctypes.byref(j), o.data_ptr(), _ptr(hh),
                                               *_shape(x.shape), dt, st), "block_join_fwd")
        return o, hh

    return _call(x.device, stream, ins + (rng,), body)


def block_join_bwd(x, m, dout, dh, gate=None, scale=None, w_post=None, w_pre=None, gate_act: str = "sigmoid",
                   eps: float = 1e-6, p: float = 0.0, rng=None, workspace=None, stream=None) -> dict:
    """Gradients of block_join_fwd for those of out and h (either may be None:
    zero), as a dict of dx, dm, dgate, dscale, dw_post and dw_pre (None where
    the input is)."""
    dt, j = _join(x, m, gate, scale, w_post, w_pre, gate_act, eps, p, rng)
    _like(dout, "dout", x, optional=True)
    _like(dh, "dh", x, optional=True)
    if dh is not None and w_pre is None:
        raise ValueError("dh goes with w_pre")

    def body(st):
        lib, shape = get_lib(), _shape(x.shape)
        g = {"dx": torch.empty_like(x), "dm": torch.empty_like(x)}
        for k, t in (("dgate", gate), ("dscale", scale), ("dw_post", w_post), ("dw_pre", w_pre)):
            g[k] = None if t is None else torch.empty_like(t)
        ws, nb = _ws(workspace, "block_join_bwd", lib.hyenand_block_join_bwd_workspace_bytes(*shape, dt), x.device, st)
        gs = _JoinGrads(*(_ptr(t) for t in g.values()))  # the structure's own order
        _done(lib.hyenand_block_join_bwd(x.data_ptr(), m.data_ptr(), ctypes.byref(j), _ptr(dout), _ptr(dh),
                                         ctypes.byref(gs), *shape, dt, ws.data_ptr(), nb, st), "block_join_bwd")
        return g

    return _call(x.device, stream, (x, m, dout, dh, gate, scale, w_post, w_pre, rng), body)


class BlockJoinFunction(torch.autograd.Function):
    """block_join_fwd and its backward as one differentiable operation; keeps
    its inputs alone (dropout's mask is drawn again from rng, which must not
    have been changed in place)."""

    @staticmethod
    def forward(ctx, x, m, gate, scale, w_post, w_pre, gate_act, eps, p, rng):
        ctx.kw = dict(gate_act=gate_act, eps=eps, p=p)
        ctx.save_for_backward(x, m, gate, scale, w_post, w_pre, rng)
        ctx.set_materialize_grads(False)
        return block_join_fwd(x, m, gate, scale, w_post, w_pre, rng=rng, **ctx.kw)

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dh):
        x, m, gate, scale, w_post, w_pre, rng = ctx.saved_tensors
        dout = None if dout is None else dout.contiguous()
        dh = None if dh is None else dh.contiguous()
        g = block_join_bwd(x, m, dout, dh, gate, scale, w_post, w_pre, rng=rng, **ctx.kw)
        return (g["dx"], g["dm"], g["dgate"], g["dscale"], g["dw_post"], g["dw_pre"], None, None, None, None)


def block_join(x, m, gate=None, scale=None, w_post=None, w_pre=None, gate_act: str = "sigmoid", eps: float = 1e-6,
               p: float = 0.0, rng=None):
    """Differentiable join (BlockJoinFunction): (out, h), h None without w_pre."""
    return BlockJoinFunction.apply(x, m, gate, scale, w_post, w_pre, gate_act, eps, p, rng)


# ------------------------------------------------------------------- dropout

def dropout_fwd(x, p: float, rng, y=None, stream=None):
    """y = x / (1 - p) where kept, else 0; x of any shape, contiguous."""
    if not isinstance(x, torch.Tensor) or not x.is_cuda or not x.is_contiguous():
        raise TypeError("x must be a contiguous device tensor")
    dt = _dtype_code(x.dtype)
    p = _rng(rng, p, x.device)

    def body(st):
        o = _out(y, "y", x, (x,))
        _done(get_lib().hyenand_dropout(x.data_ptr(), o.data_ptr(), x.numel(), dt, p, _ptr(rng) if p else None, st),
              "dropout")
        return o

    return _call(x.device, stream, (x, rng), body)


def dropout_bwd(dy, p: float, rng, dx=None, stream=None):
    """dx of dropout_fwd: the same mask and factor on the gradient dy."""
    return dropout_fwd(dy, p, rng, y=dx, stream=stream)


class DropoutFunction(torch.autograd.Function):
    """dropout_fwd and its backward as one differentiable operation; keeps rng
    alone, which must not have been changed in place."""

    @staticmethod
    def forward(ctx, x, p, rng):
        ctx.p = p
        ctx.save_for_backward(rng)
        return dropout_fwd(x, p, rng)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        (rng,) = ctx.saved_tensors
        return dropout_bwd(dy.contiguous(), ctx.p, rng), None, None


def dropout(x, p: float, rng):
    """Differentiable dropout without a stored mask (DropoutFunction)."""
    return DropoutFunction.apply(x, p, rng)


# -------------------------------------------------------------- feed-forward

def _ffn(x, Wg, Wu, Wd, act):
    dt = _x(x)
    C = int(x.shape[1])
    F = int(Wg.shape[0]) if isinstance(Wg, torch.Tensor) and Wg.dim() == 2 else -1
    for t, nm, shape in ((Wg, "Wg", (F, C)), (Wu, "Wu", (F, C)), (Wd, "Wd", (C, F))):
        if not isinstance(t, torch.Tensor) or t.dtype != x.dtype or t.device != x.device or not t.is_contiguous():
            raise TypeError(f"{nm} must be a contiguous {x.dtype} tensor on {x.device}")
        if tuple(t.shape) != shape:
            raise ValueError(f"{nm} must have the shape {shape}, got {tuple(t.shape)}")
    return dt, F, _act(act, ("sigmoid", "silu", "gelu"))


def gated_ffn_workspace_bytes(B: int, C: int, F: int, dims, dtype=torch.float32) -> int:
    return int(get_lib().hyenand_gated_ffn_workspace_bytes(B, C, F, len(dims), _dims_arr(dims), _dtype_code(dtype)))


def gated_ffn_bwd_workspace_bytes(B: int, C: int, F: int, dims, dtype=torch.float32) -> int:
    return int(get_lib().hyenand_gated_ffn_bwd_workspace_bytes(B, C, F, len(dims), _dims_arr(dims),
                                                               _dtype_code(dtype)))


def gated_ffn_fwd(x, Wg, Wu, Wd, act: str = "silu", y=None, workspace=None, stream=None):
    """y = Wd (act(Wg x) * (Wu x)) at every position; Wg, Wu [F, C], Wd [C, F]
    of x's dtype, 16-byte aligned like x."""
    dt, F, a = _ffn(x, Wg, Wu, Wd, act)

    def body(st):
        lib, (B, C, d, dims) = get_lib(), _shape(x.shape)
        o = _out(y, "y", x, (x, Wg, Wu, Wd))
        ws, nb = _ws(workspace, "gated_ffn", lib.hyenand_gated_ffn_workspace_bytes(B, C, F, d, dims, dt), x.device, st)
        _done(lib.hyenand_gated_ffn_fwd(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(), o.data_ptr(), B, C, F,
                                        d, dims, dt, a, ws.data_ptr(), nb, st), "gated_ffn_fwd")
        return o

    return _call(x.device, stream, (x, Wg, Wu, Wd), body)


def gated_ffn_bwd(x, Wg, Wu, Wd, dy, act: str = "silu", workspace=None, stream=None):
    """(dx, dWg, dWu, dWd) of gated_ffn_fwd for the gradient dy of y."""
    dt, F, a = _ffn(x, Wg, Wu, Wd, act)
    _like(dy, "dy", x)

    def body(st):
        lib, (B, C, d, dims) = get_lib(), _shape(x.shape)
        dx, dWg, dWu, dWd = (torch.empty_like(t) for t in (x, Wg, Wu, Wd))
        ws, nb = _ws(workspace, "gated_ffn_bwd", lib.hyenand_gated_ffn_bwd_workspace_bytes(B, C, F, d, dims, dt),
                     x.device, st)
        _done(lib.hyenand_gated_ffn_bwd(x.data_ptr(), Wg.data_ptr(), Wu.data_ptr(), Wd.data_ptr(), dy.data_ptr(),
                                        dx.data_ptr(), dWg.data_ptr(), dWu.data_ptr(), dWd.data_ptr(), B, C, F, d, dims,
                                        dt, a, ws.data_ptr(), nb, st), "gated_ffn_bwd")
        return dx, dWg, dWu, dWd

    return _call(x.device, stream, (x, Wg, Wu, Wd, dy), body)


class GatedFFNFunction(torch.autograd.Function):
    """gated_ffn_fwd and its backward as one differentiable operation; keeps
    its inputs alone and recomputes the hidden values in the backward, as the
    convolution's does with its transforms."""

    @staticmethod
    def forward(ctx, x, Wg, Wu, Wd, act):
        ctx.act = act
        ctx.save_for_backward(x, Wg, Wu, Wd)
        return gated_ffn_fwd(x, Wg, Wu, Wd, act)

    @staticmethod
    @once_differentiable
    def backward(ctx, dy):
        dy = dy.contiguous()
        if dy.data_ptr() % 16:  # part of a larger gradient
            dy = dy.clone()
        dx, dWg, dWu, dWd = gated_ffn_bwd(*ctx.saved_tensors, dy, ctx.act)
        return dx, dWg, dWu, dWd, None


def gated_ffn(x, Wg, Wu, Wd, act: str = "silu"):
    """Differentiable gated feed-forward block (GatedFFNFunction)."""
    return GatedFFNFunction.apply(x, Wg, Wu, Wd, act)
