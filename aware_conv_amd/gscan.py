"""Binding of the gated linear recurrence (include/gscan.h) and its autograd
function.

Activations are ``[B, C, T]`` (``layout="bct"``; also ``[B, C, H, W]`` planes,
taken in raster order) or ``[B, T, C]`` (``layout="btc"``), in float32, float16
or bfloat16.  Elements along the last axis are adjacent; the other strides are
free, so that x and the gates may be chunks of one projection.
"""
import ctypes
import functools

import torch

from . import _lib

try:
    from . import _lists
except ImportError as e:
    raise ImportError("_lists.so is not built (%s); run `python -m aware_conv_amd.build` or "
                      "__graft_entry__.build() first" % e)

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
LAYOUTS = {"bct": 0, "btc": 1}
GRAD_NAMES = ("dx", "dr", "di", "dlam", "dh0")
MAX_T = 1 << 30


def _dtype_code(t):
    if t.dtype not in DTYPES:
        raise TypeError("the recurrence supports float32, float16 and bfloat16 tensors, got %s"
                        % t.dtype)
    return DTYPES[t.dtype]


def _rows_and_run(shape, layout):
    """Dimensions of an activation as (B, C, T)."""
    if layout not in LAYOUTS:
        raise ValueError("layout must be 'bct' or 'btc', got %r" % (layout,))
    if layout == "btc":
        if len(shape) != 3:
            raise ValueError("activations must be [B, T, C], got shape %s" % (tuple(shape),))
        return shape[0], shape[2], shape[1]
    if len(shape) not in (3, 4):
        raise ValueError("activations must be [B, C, T] or [B, C, H, W], got shape %s"
                         % (tuple(shape),))
    return shape[0], shape[1], shape[2] * (shape[3] if len(shape) == 4 else 1)


def _adjacent(t):
    """Whether a row of `t` (its last axis, or the planes of a 4-D tensor) is one run."""
    if t.is_contiguous() or t.numel() == 0:
        return True
    shape, st = t.shape, t.stride()
    if len(shape) == 4 and not (shape[2] == 1 or st[2] == shape[3]):
        return False
    return shape[-1] == 1 or st[-1] == 1


# Tensors are checked and read by a small extension (pyext/tensor_lists.cpp);
# what it refuses is looked at again here, to say what is wrong.

def _refuse(names, tensors, flats):
    """Raises what is wrong with the activations `tensors` (that go by the first, or None) or the
    contiguous tensors `flats` ((name, tensor, dtype, n0, n1 or -1)): shapes first, devices last."""
    x = tensors[0]
    for name, t in zip(names, tensors):
        if t is None and t is not x and name in _MAY_LACK:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if t.shape != x.shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(x.shape)))
        if t.dtype is not x.dtype:
            raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, x.dtype))
        if not _adjacent(t):
            raise ValueError("%s must have adjacent elements along its rows" % name)
    for name, t, dtype, n0, n1 in flats:
        if t is None and name in _MAY_LACK:
            continue
        _lib._expect(dtype, [(name, t, (n0,) if n1 < 0 else (n0, n1))])
        if t is None:
            raise TypeError("%s must be a torch.Tensor" % name)
    _lib._on_gpu(x, list(zip(names, tensors)) + [f[:2] for f in flats])
    raise ValueError("tensors of an unsupported kind")


_MAY_LACK = {"h0", "lengths", "dh_last", "slots", "h"} | {"grads[%s]" % n for n in GRAD_NAMES}
_f32, _i32 = torch.float32, torch.int32
_VIEW = ctypes.sizeof(_lib.GscanView)
_Views4, _Views7 = _lib.GscanView * 4, _lib.GscanView * 7


def _view(t):
    return t.data_ptr(), t.stride(0), t.stride(1)


def _read(out, names, tensors, flats):
    """(address of the views of `tensors` in `out`, addresses of `flats`), checked."""
    at = ctypes.addressof(out)
    bad = _lists.views(tensors, at) >= 0
    device = tensors[0].device.index
    if not bad:
        ps = [_lists.flat(t, dtype, device, n0, n1) for _, t, dtype, n0, n1 in flats]
        # None only where one may lack
        bad = any(p is False or (p is None and f[0] not in _MAY_LACK) for p, f in zip(ps, flats))
        # an activation that lacks and may not
        bad = bad or any(t is None and n not in _MAY_LACK for n, t in zip(names, tensors))
    if bad:
        _refuse(names, tensors, flats)
    return at, ps


def _input(x):
    """(dtype code, dtype, device) of the tensor that the others go by."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    return _dtype_code(x), x.dtype, x.device


def on_stream(call):
    """A call given a stream that is not the current one runs with it as the current one: what it
    allocates then belongs to that stream, and is not handed out again while its kernels use it."""
    @functools.wraps(call)
    def wrapped(*args, **kw):
        stream = kw.get("stream")
        if stream is None:
            return call(*args, **kw)
        with torch.cuda.stream(stream):
            return call(*args, **kw)
    return wrapped


def _raw_stream(stream, device):
    """The handle of a stream, which must be on the tensors' device; without one, that of the
    device's current stream, as an integer (a Stream object would cost as much as the rest of a
    small call's marshalling)."""
    if stream is None:
        return torch._C._cuda_getCurrentRawStream(device.index)
    if stream.device != device:
        raise ValueError("stream is on %s; every tensor is on %s" % (stream.device, device))
    return stream.cuda_stream


@functools.lru_cache(maxsize=256)
def _sizes(B, C, T, layout, code):
    """(floats of the states, bytes of the workspace) for a shape."""
    s = _lib.GscanShape(B, C, T, layout, code, 0, 1.0)
    out = []
    for fn in ("gscan_states_size", "gscan_workspace_size"):
        n = ctypes.c_size_t(0)
        _lib._check(getattr(_lib.lib, fn)(ctypes.byref(s), ctypes.byref(n)), fn)
        out.append(n.value)
    return out[0] // 4, out[1]


def _shape(x, code, layout, reverse, decay):
    B, C, T = _rows_and_run(x.shape, layout)
    if T > MAX_T:
        raise ValueError("at most %d positions are supported, got %d" % (MAX_T, T))
    return _lib.GscanShape(B, C, T, LAYOUTS[layout], code, 1 if reverse else 0, decay)


def _workspace(s, device, workspace):
    """(tensor, address, bytes); the caller keeps the tensor until the call was enqueued."""
    if workspace is None:
        need = _sizes(s.B, s.C, s.T, s.layout, s.dtype)[1]
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    elif workspace.device != device:
        raise ValueError("workspace is on %s; every tensor must be on %s" % (workspace.device, device))
    return workspace, workspace.data_ptr(), workspace.numel() * workspace.element_size()


def gscan_workspace_size(x, layout="bct"):
    """Bytes of workspace gscan_fwd and gscan_bwd need for activations like x."""
    B, C, T = _rows_and_run(x.shape, layout)
    return _sizes(B, C, T, LAYOUTS[layout], _dtype_code(x))[1]


@on_stream
def gscan_fwd(x, r, i, lam, h0=None, lengths=None, layout="bct", reverse=False, decay=8.0, h=None,
              save_states=False, workspace=None, *, stream=None):
    """(h, h_last, states) of the recurrence: h like x, h_last [B, C] fp32 the state after the
    last valid position, states what gscan_bwd needs (None unless ``save_states``).  lam [C] and
    h0 [B, C] are fp32, lengths [B] int32 (see include/gscan.h)."""
    code, dt, dev = _input(x)
    s = _shape(x, code, layout, reverse, decay)
    v = _Views4()
    B, C = s.B, s.C
    p, (plam, ph0, plen) = _read(v, ("x", "r", "i", "h"), (x, r, i, h),
                                 (("lam", lam, _f32, C, -1), ("h0", h0, _f32, B, C),
                                  ("lengths", lengths, _i32, B, -1)))
    given = h
    if h is None:
        h = torch.empty(x.shape, dtype=dt, device=dev)
        v[3] = _view(h)
    h_last = torch.empty((B, C), dtype=_f32, device=dev)
    states = pstates = None
    if save_states:
        states = torch.empty(_sizes(s.B, s.C, s.T, s.layout, code)[0], dtype=_f32, device=dev)
        pstates = states.data_ptr()
    ws, pws, nws = _workspace(s, dev, workspace)
    _lib._enqueue(dev, "gscan_fwd", ctypes.byref(s), p, p + _VIEW, p + 2 * _VIEW, plam, ph0, plen,
                  p + 3 * _VIEW, h_last.data_ptr(), pstates, pws, nws, _raw_stream(stream, dev))
    if given is not None:
        _lists.written(given)
    return h, h_last, states


@on_stream
def gscan_bwd(x, r, i, lam, states, dh, dh_last=None, lengths=None, layout="bct", reverse=False,
              decay=8.0, grads=None, workspace=None, *, stream=None):
    """Gradients of <dh, h> + <dh_last, h_last> as a dict keyed by GRAD_NAMES, from the inputs
    and the states of gscan_fwd.  ``grads`` may hold tensors to write (dx, dr, di with free
    strides); those it lacks are allocated."""
    given = tuple((grads or {}).values())
    grads = dict(grads or {})
    unknown = [n for n in grads if n not in GRAD_NAMES]
    if unknown:
        raise KeyError("unknown gradients %s" % ", ".join(map(str, unknown)))
    code, dt, dev = _input(x)
    s = _shape(x, code, layout, reverse, decay)
    names = ("dx", "dr", "di")
    v = _Views7()
    B, C = s.B, s.C
    if states is None:
        raise ValueError("gscan_bwd needs the states of gscan_fwd(..., save_states=True)")
    p, (plam, plast, plen, pdlam, pdh0, pst) = _read(
        v, ("x", "r", "i", "dh", "grads[dx]", "grads[dr]", "grads[di]"),
        (x, r, i, dh, *[grads.get(n) for n in names]),
        (("lam", lam, _f32, C, -1), ("dh_last", dh_last, _f32, B, C), ("lengths", lengths, _i32, B, -1),
         ("grads[dlam]", grads.get("dlam"), _f32, C, -1), ("grads[dh0]", grads.get("dh0"), _f32, B, C),
         ("states", states, _f32, _sizes(B, C, s.T, s.layout, code)[0], -1)))
    for k, n in enumerate(names):
        if grads.get(n) is None:
            grads[n] = torch.empty(x.shape, dtype=dt, device=dev)
            v[4 + k] = _view(grads[n])
    if pdlam is None:
        grads["dlam"] = torch.empty(C, dtype=_f32, device=dev)
        pdlam = grads["dlam"].data_ptr()
    if pdh0 is None:
        grads["dh0"] = torch.empty((B, C), dtype=_f32, device=dev)
        pdh0 = grads["dh0"].data_ptr()
    ws, pws, nws = _workspace(s, dev, workspace)
    _lib._enqueue(dev, "gscan_bwd", ctypes.byref(s), p, p + _VIEW, p + 2 * _VIEW, plam, pst, plen,
                  p + 3 * _VIEW, plast, p + 4 * _VIEW, p + 5 * _VIEW, p + 6 * _VIEW, pdlam, pdh0,
                  pws, nws, _raw_stream(stream, dev))
    _lists.written(given)
    return grads


@on_stream
def gscan_step(x, r, i, lam, state, slots=None, decay=8.0, h=None, *, stream=None):
    """One position of B sequences: x, r, i [B, C] (free row strides), their states in rows
    ``slots`` (int32 [B]; the first B rows if None) of ``state`` [S, C] fp32, which is updated.
    Returns h [B, C].  Sequences whose slot is outside 0..S-1 give zeros and change nothing."""
    code, dt, dev = _input(x)
    if x.dim() != 2:
        raise ValueError("activations must be [B, C], got shape %s" % (tuple(x.shape),))
    B, C = x.shape
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be a torch.Tensor")
    if state.dim() != 2 or state.shape[1] != C:
        raise ValueError("state must be [S, %d], got shape %s" % (C, tuple(state.shape)))
    S = state.shape[0]
    if slots is None and S < B:
        raise ValueError("state has %d rows for %d sequences" % (S, B))
    v = _Views4()
    p, (plam, pstate, pslots) = _read(v, ("x", "r", "i", "h"), (x, r, i, h),
                                      (("lam", lam, _f32, C, -1), ("state", state, _f32, S, C),
                                       ("slots", slots, _i32, B, -1)))
    given = h
    if h is None:
        h = torch.empty((B, C), dtype=dt, device=dev)
        v[3] = _view(h)
    _lib._enqueue(dev, "gscan_step", B, C, S, code, decay, p, p + _VIEW, p + 2 * _VIEW, plam,
                  pstate, pslots, p + 3 * _VIEW, _raw_stream(stream, dev))
    _lists.written(state, given)
    return h


def _rows(t):
    return t if _adjacent(t) else t.contiguous()


class GatedScanFunction(torch.autograd.Function):
    """Forward through ``gscan_fwd``, backward through ``gscan_bwd``.  Saved are the inputs and
    the states the tiles start from; the outputs are formed again by the backward kernel."""

    @staticmethod
    def forward(ctx, x, r, i, lam, h0, lengths, layout, reverse, decay):
        x, r, i = _rows(x), _rows(r), _rows(i)
        lam = lam.contiguous()
        h0 = None if h0 is None else h0.contiguous()
        want = any(ctx.needs_input_grad[:5])
        h, h_last, states = gscan_fwd(x, r, i, lam, h0=h0, lengths=lengths, layout=layout,
                                      reverse=reverse, decay=decay, save_states=want)
        if want:
            ctx.save_for_backward(x, r, i, lam, lengths, states)
            ctx.form = {"layout": layout, "reverse": reverse, "decay": decay}
        return h, h_last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dh, dh_last):
        x, r, i, lam, lengths, states = ctx.saved_tensors
        if dh is None:
            dh = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        g = gscan_bwd(x, r, i, lam, states, _rows(dh), lengths=lengths,
                      dh_last=None if dh_last is None else dh_last.contiguous(), **ctx.form)
        out = [g[n] if need else None for n, need in zip(GRAD_NAMES, ctx.needs_input_grad)]
        return (*out, None, None, None, None)


def gated_scan(x, r, i, lam, h0=None, lengths=None, layout="bct", reverse=False, decay=8.0):
    """(h, h_last) of the gated linear recurrence, differentiable in x, r, i, lam and h0."""
    return GatedScanFunction.apply(x, r, i, lam, h0, lengths, layout, reverse, decay)
