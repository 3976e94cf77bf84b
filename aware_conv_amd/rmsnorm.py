"""Binding of the root-mean-square norm with the residual's addition (include/rmsnorm.h) and its
autograd function.

Rows are the last axis of ``[B, T, C]`` or ``[B, C]`` tensors in float32, float16 or bfloat16,
whose elements are adjacent; the other strides are free.  The residual stream is of the same type
or float32, the weight float32."""
import ctypes
import functools

import torch

from . import _acts, _lib, gscan
from ._acts import VIEW, f32
from .gscan import _lists, _raw_stream, on_stream

GRAD_NAMES = ("dx", "dresidual", "dw")
MAX_C = 1 << 20
_Views4, _Views5 = _lib.GscanView * 4, _lib.GscanView * 5


@functools.lru_cache(maxsize=256)
def _form(*shape):
    """The shape as the library takes it; it is only read."""
    return ctypes.byref(_lib.RmsnormShape(*shape))


@functools.lru_cache(maxsize=256)
def _need(*shape):
    """Bytes of the backward's workspace for a shape."""
    s, n = _lib.RmsnormShape(*shape), ctypes.c_size_t(0)
    _lib._check(_lib.lib.rmsnorm_workspace_size(ctypes.byref(s), ctypes.byref(n)), "rmsnorm_workspace_size")
    return n.value


def _shape(x, name="x"):
    """(B, T, C, dtype code) of the tensor that the others go by."""
    code = gscan._dtype_code(_acts.tensor(name, x))
    if x.dim() not in (2, 3):
        raise ValueError("%s must be [B, T, C] or [B, C], got shape %s" % (name, tuple(x.shape)))
    size = x.shape
    if size[-1] > MAX_C:
        raise ValueError("rows of at most %d elements are supported, got %d" % (MAX_C, size[-1]))
    return size[0], size[1] if len(size) == 3 else 1, size[-1], code


def _stream_code(x, code, name, t):
    """The dtype code of the residual stream, which is x's or float32."""
    if _acts.tensor(name, t).dtype is not x.dtype and t.dtype is not f32:
        raise TypeError("%s has dtype %s, expected %s or torch.float32" % (name, t.dtype, x.dtype))
    if t.shape != x.shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(x.shape)))
    return code if t.dtype is x.dtype else 0


def _put(v, k, t):
    v[k] = (t.data_ptr(), t.stride(0), t.stride(1))


def rmsnorm_workspace_size(x):
    """Bytes of workspace rmsnorm_bwd needs for rows like x."""
    B, T, C, code = _shape(x)
    return _need(B, T, C, code, code, 0.0)


def _forward(x, w, residual, eps, y, total, scale, save_rstd, stream, e4m3):
    B, T, C, code = _shape(x)
    if residual is None and total is not None:
        raise ValueError("total is given without a residual")
    rcode = code if residual is None else _stream_code(x, code, "residual", residual)
    v = _Views4()  # x, y, residual, total
    rows = x.shape[:-1]
    p, (pw, pscale) = _acts.read(
        v, x, ((("x", "y"), (x, None if e4m3 else y)), (("residual", "total"), (residual, total))),
        (("w", w, f32, (C,), False), ("scale", scale, f32, rows, True)))
    dev = x.device
    given = [t for t in (y, total, scale) if t is not None]
    if e4m3 and y is not None:
        if _acts.tensor("y", y).dtype is not torch.float8_e4m3fn:
            raise TypeError("y has dtype %s, expected torch.float8_e4m3fn" % y.dtype)
        if y.shape != x.shape or not gscan._adjacent(y) or y.device != dev:
            raise ValueError("y must be like x, with adjacent elements along its rows, on %s" % dev)
        _put(v, 1, y)
    if y is None:
        y = torch.empty(x.shape, dtype=torch.float8_e4m3fn, device=dev) if e4m3 else _acts.like(x)
        v[1] = y.data_ptr(), T * C, C
    if residual is not None and total is None:
        total = _acts.like(residual)
        v[3] = total.data_ptr(), T * C, C
    if e4m3 and scale is None:
        scale = torch.empty(rows, dtype=f32, device=dev)
        pscale = scale.data_ptr()
    rstd = torch.empty(rows, dtype=f32, device=dev) if save_rstd else None
    there = residual is not None
    args = (p, p + 2 * VIEW if there else None, pw, p + VIEW, *((pscale,) if e4m3 else ()),
            p + 3 * VIEW if there else None, None if rstd is None else rstd.data_ptr(), _raw_stream(stream, dev))
    _lib._enqueue(dev, "rmsnorm_fwd_e4m3" if e4m3 else "rmsnorm_fwd", _form(B, T, C, code, rcode, eps), *args)
    if given:
        _lists.written(given)
    return y, total, scale, rstd


@on_stream
def rmsnorm_fwd(x, w, residual=None, eps=1e-6, y=None, total=None, save_rstd=False, *, stream=None):
    """(y, total, rstd): y like x the norm of total = x + residual (of x, and total is None, without
    a residual), rstd [B, T] what rmsnorm_bwd needs (None unless ``save_rstd``).  w [C] is fp32;
    total may be the residual itself, which is then updated (see include/rmsnorm.h)."""
    y, total, _, rstd = _forward(x, w, residual, eps, y, total, None, save_rstd, stream, False)
    return y, total, rstd


@on_stream
def rmsnorm_fwd_e4m3(x, w, residual=None, eps=1e-6, y=None, total=None, scale=None, *, stream=None):
    """(y, scale, total): rmsnorm_fwd with y in torch.float8_e4m3fn, to be multiplied by scale [B, T]
    (one number per row)."""
    y, total, scale, _ = _forward(x, w, residual, eps, y, total, scale, False, stream, True)
    return y, scale, total


@on_stream
def rmsnorm_bwd(kept, w, rstd, dy, dtotal=None, grads=None, workspace=None, *, stream=None):
    """Gradients of <dy, y> + <dtotal, total> as a dict keyed by GRAD_NAMES, from what was normed
    (``kept``: total, or x without a residual) and rstd.  dx is of dy's type; dresidual of kept's,
    and dx itself where these are the same.  ``grads`` may hold tensors to write (dx, dresidual
    with free strides); those it lacks are allocated."""
    given = tuple((grads or {}).values())
    grads = _acts.known(grads, GRAD_NAMES)
    B, T, C, code = _shape(dy, "dy")
    rcode = _stream_code(dy, code, "kept", kept)
    two, get = rcode != code, grads.get
    if not two and get("dresidual") is not None:
        raise ValueError("grads[dresidual] is grads[dx], which is of the same type")
    v = _Views5()  # dy, dx, kept, dtotal, dresidual
    p, (pw, prstd, pdw) = _acts.read(
        v, dy, ((("dy", "grads[dx]"), (dy, get("dx"))),
                (("kept", "dtotal", "grads[dresidual]"), (kept, dtotal, get("dresidual")))),
        (("w", w, f32, (C,), False), ("rstd", rstd, f32, dy.shape[:-1], False),
         ("grads[dw]", get("dw"), f32, (C,), True)))
    dev = dy.device
    if get("dx") is None:
        grads["dx"] = _acts.like(dy)
        _put(v, 1, grads["dx"])
    if two and get("dresidual") is None:
        grads["dresidual"] = _acts.like(kept)
        _put(v, 4, grads["dresidual"])
    if pdw is None:
        grads["dw"] = torch.empty(C, dtype=f32, device=dev)
        pdw = grads["dw"].data_ptr()
    ws, pws, nws = _acts.workspace(_need(B, T, C, code, rcode, 0.0), dev, workspace)
    _lib._enqueue(dev, "rmsnorm_bwd", _form(B, T, C, code, rcode, 0.0), p + 2 * VIEW, pw,
                  prstd, p, None if dtotal is None else p + 3 * VIEW, p + VIEW, p + 4 * VIEW if two else None, pdw,
                  pws, nws, _raw_stream(stream, dev))
    _lists.written(given)
    if not two:
        grads["dresidual"] = grads["dx"]
    return {n: grads[n] for n in GRAD_NAMES}


class RmsNormFunction(torch.autograd.Function):
    """Forward through ``rmsnorm_fwd``, backward through ``rmsnorm_bwd``.  Saved are the sum that was
    normed and a number per row."""

    @staticmethod
    def forward(ctx, x, w, residual, eps):
        ctx.set_materialize_grads(False)
        x, w, residual = _acts.rows(x), _acts.flat(w), _acts.rows(residual)
        want = any(ctx.needs_input_grad[:3])
        y, total, rstd = rmsnorm_fwd(x, w, residual=residual, eps=eps, save_rstd=want)
        if want:
            ctx.save_for_backward(x if total is None else total, w, rstd)
            ctx.dtype = x.dtype
        return y, total

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dtotal):
        kept, w, rstd = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(kept.shape, dtype=ctx.dtype, device=kept.device)
        g = rmsnorm_bwd(kept, w, rstd, _acts.rows(dy), dtotal=_acts.rows(dtotal))
        need = ctx.needs_input_grad
        return (g["dx"] if need[0] else None, g["dw"] if need[1] else None,
                g["dresidual"] if need[2] else None, None)


def rms_norm(x, w, residual=None, eps=1e-6):
    """(y, total) of the root-mean-square norm, differentiable in x, w and residual; total is None
    without a residual."""
    return RmsNormFunction.apply(x, w, residual, eps)
