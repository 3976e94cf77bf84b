"""Binding of the short causal convolution (include/cconv.h) and its autograd function.

Activations are token sequences ``[B, T, C]`` in float32, float16 or bfloat16.  Channels are
adjacent; the other strides are free, so that they may be parts of projections.  The inputs kept
of a sequence (``h0``, ``last``, a cache's rows) are ``[B, K - 1, C]`` of the activations' type,
weights and their gradients float32."""
import ctypes
import functools

import torch

from . import _acts, _lib, gscan
from ._acts import VIEW, f32, i32
from .gscan import _lists, _raw_stream, _view, on_stream

GRAD_NAMES = ("dx", "dw", "dbias", "dh0")
MAX_T = 1 << 30
MAX_TAPS = 8
_Views2, _Views3 = _lib.GscanView * 2, _lib.GscanView * 3


@functools.lru_cache(maxsize=256)
def _form(*shape):
    """The shape as the library takes it; it is only read."""
    return ctypes.byref(_lib.CconvShape(*shape))


@functools.lru_cache(maxsize=256)
def _need(*shape):
    """Bytes of the backward's workspace for a shape."""
    s, n = _lib.CconvShape(*shape), ctypes.c_size_t(0)
    _lib._check(_lib.lib.cconv_workspace_size(ctypes.byref(s), ctypes.byref(n)), "cconv_workspace_size")
    return n.value


def _shape(x, w, silu, axes):
    """(B, T, C, K, dtype code, silu) from the tensors that the others go by."""
    code = gscan._dtype_code(_acts.tensor("x", x))
    size = _acts.dims("x", x, axes, "[B, T, C]" if axes == 3 else "[B, C]")
    T = size[1] if axes == 3 else 1
    if T > MAX_T:
        raise ValueError("at most %d positions are supported, got %d" % (MAX_T, T))
    n = _acts.dims("w", w, 2, "[C, K]")
    if n[0] != size[-1] or not 1 <= n[1] <= MAX_TAPS:
        raise ValueError("w has shape %s, expected [%d, K] with K of 1 to %d" % (tuple(n), size[-1], MAX_TAPS))
    return size[0], T, size[-1], n[1], code, 1 if silu else 0


def cconv_workspace_size(x, w):
    """Bytes of workspace cconv_bwd needs for tensors like these."""
    return _need(*_shape(x, w, True, 3))


@on_stream
def cconv_fwd(x, w, bias=None, h0=None, lengths=None, silu=True, y=None, *, stream=None):
    """(y, last): y like x, last [B, K - 1, C] the inputs from which the sequence can be continued.
    w [C, K] and bias [C] are fp32, h0 [B, K - 1, C] (the inputs before the first; zeros if None)
    of x's type, lengths [B] int32 (see include/cconv.h)."""
    shape = B, T, C, K, code, _ = _shape(x, w, silu, 3)
    v = _Views2()
    p, (pw, pb, ph0, plen) = _acts.read(
        v, x, ((("x", "y"), (x, y)),),
        (("w", w, f32, (C, K), False), ("bias", bias, f32, (C,), True), ("h0", h0, x.dtype, (B, K - 1, C), True),
         ("lengths", lengths, i32, (B,), True)))
    dev, given = x.device, y
    if y is None:
        y = _acts.like(x)
        v[1] = _view(y)
    last = torch.empty((B, K - 1, C), dtype=x.dtype, device=dev)
    _lib._enqueue(dev, "cconv_fwd", _form(*shape), p, pw, pb, ph0, plen, p + VIEW,
                  last.data_ptr(), _raw_stream(stream, dev))
    if given is not None:
        _lists.written(given)
    return y, last


@on_stream
def cconv_bwd(x, w, dy, bias=None, h0=None, dlast=None, lengths=None, silu=True, grads=None, workspace=None, *,
              stream=None):
    """Gradients of <dy, y> + <dlast, last> as a dict keyed by GRAD_NAMES, from the inputs of
    cconv_fwd; dbias is there where bias is.  ``grads`` may hold tensors to write (dx with free
    strides); those it lacks are allocated."""
    given = tuple((grads or {}).values())
    grads = _acts.known(grads, GRAD_NAMES)
    shape = B, T, C, K, code, _ = _shape(x, w, silu, 3)
    if bias is None and grads.get("dbias") is not None:
        raise ValueError("grads[dbias] is given without bias")
    v, get, kept = _Views3(), grads.get, (B, K - 1, C)
    p, (pw, pb, ph0, plen, plast, pdw, pdb, pdh0) = _acts.read(
        v, x, ((("x", "dy", "grads[dx]"), (x, _acts.tensor("dy", dy), get("dx"))),),
        (("w", w, f32, (C, K), False), ("bias", bias, f32, (C,), True), ("h0", h0, x.dtype, kept, True),
         ("lengths", lengths, i32, (B,), True), ("dlast", dlast, x.dtype, kept, True),
         ("grads[dw]", get("dw"), f32, (C, K), True), ("grads[dbias]", get("dbias"), f32, (C,), True),
         ("grads[dh0]", get("dh0"), x.dtype, kept, True)))
    dev = x.device
    if get("dx") is None:
        grads["dx"] = _acts.like(x)
        v[2] = _view(grads["dx"])
    out = []
    for n, at, size, dtype, there in (("dw", pdw, (C, K), f32, True), ("dbias", pdb, (C,), f32, bias is not None),
                                      ("dh0", pdh0, kept, x.dtype, True)):
        if at is None and there:
            grads[n] = torch.empty(size, dtype=dtype, device=dev)
            at = grads[n].data_ptr()
        out.append(at)
    ws, pws, nws = _acts.workspace(_need(*shape), dev, workspace)
    _lib._enqueue(dev, "cconv_bwd", _form(*shape), p, pw, pb, ph0, plen, p + VIEW, plast,
                  p + 2 * VIEW, out[0], out[1], out[2], pws, nws, _raw_stream(stream, dev))
    _lists.written(given)
    return {n: grads.get(n) for n in GRAD_NAMES}


@on_stream
def cconv_step(x, w, cache, bias=None, slots=None, silu=True, y=None, *, stream=None):
    """One position of B sequences: x [B, C] (free row stride), their last inputs in rows ``slots``
    (int32 [B]; the first B rows if None) of ``cache`` [S, K - 1, C], which is moved on.  Returns y
    [B, C].  Sequences whose slot is outside 0..S-1 give zeros and change nothing."""
    shape = B, _, C, K, code, _ = _shape(x, w, silu, 2)
    S = _acts.dims("cache", cache, 3, "[S, K - 1, C]")[0]
    if slots is None and S < B:
        raise ValueError("cache has %d rows for %d sequences" % (S, B))
    v = _Views2()
    p, (pw, pb, pcache, pslots) = _acts.read(
        v, x, ((("x", "y"), (x, y)),),
        (("w", w, f32, (C, K), False), ("bias", bias, f32, (C,), True),
         ("cache", cache, x.dtype, (S, K - 1, C), False), ("slots", slots, i32, (B,), True)))
    dev, given = x.device, y
    if y is None:
        y = _acts.like(x)
        v[1] = _view(y)
    _lib._enqueue(dev, "cconv_step", _form(*shape), S, p, pw, pb, pcache, pslots, p + VIEW,
                  _raw_stream(stream, dev))
    _lists.written(cache, given)
    return y


class CausalConvFunction(torch.autograd.Function):
    """Forward through ``cconv_fwd``, backward through ``cconv_bwd``.  Only inputs are saved."""

    @staticmethod
    def forward(ctx, x, w, bias, h0, lengths, silu):
        ctx.set_materialize_grads(False)
        x = _acts.rows(x)
        w, bias, h0 = (_acts.flat(t) for t in (w, bias, h0))
        ctx.save_for_backward(x, w, bias, h0, lengths)
        ctx.silu = silu
        return cconv_fwd(x, w, bias=bias, h0=h0, lengths=lengths, silu=silu)

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dlast):
        x, w, bias, h0, lengths = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        g = cconv_bwd(x, w, _acts.rows(dy), bias=bias, h0=h0, dlast=_acts.flat(dlast), lengths=lengths,
                      silu=ctx.silu)
        return (*[g[n] if need else None for n, need in zip(GRAD_NAMES, ctx.needs_input_grad)], None, None)


def causal_conv(x, w, bias=None, h0=None, lengths=None, silu=True):
    """(y, last) of the short causal convolution, differentiable in x, w, bias and h0."""
    return CausalConvFunction.apply(x, w, bias, h0, lengths, silu)
