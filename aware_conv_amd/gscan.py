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


# The checks below and the marshalling run once per call and tensor; small calls
# take about as long as they do, so each is one function per tensor that asks
# for every attribute once, and pointers go to ctypes as plain integers.

def _act(name, t, shape, dtype, device):
    """The view of an activation that is `shape`, `dtype`, on `device` and has adjacent rows."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not _adjacent(t):
        raise ValueError("%s must have adjacent elements along its rows" % name)
    if t.device != device:
        raise ValueError("%s is on %s; every tensor must be on %s" % (name, t.device, device))
    st = t.stride()
    return ctypes.byref(_View(t.data_ptr(), st[0], st[1]))


def _flat(name, t, shape, dtype, device):
    """The address of a contiguous tensor of `shape` and `dtype` on `device`; None for None."""
    if t is None:
        return None
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if shape is not None and t.shape != shape:
        raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(shape)))
    if dtype is not None and t.dtype is not dtype:
        raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, dtype))
    if not t.is_contiguous():
        raise ValueError("%s must be contiguous" % name)
    if t.device != device:
        raise ValueError("%s is on %s; every tensor must be on %s" % (name, t.device, device))
    return t.data_ptr()


_View = _lib.GscanView
_f32, _i32 = torch.float32, torch.int32


def _input(x):
    """(dtype code, dtype, device) of the tensor that the others go by."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    return _dtype_code(x), x.dtype, x.device


def _on_gpu(device):
    if device.type != "cuda":
        raise ValueError("x is on %s; every tensor must be on a GPU" % device)


def _raw_stream(stream, device):
    """The stream's handle; without a stream, that of the current one, as an integer (a Stream
    object would cost as much as the rest of a small call's marshalling)."""
    return stream.cuda_stream if stream is not None else torch._C._cuda_getCurrentRawStream(device.index)


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
    p = _flat("workspace", workspace, None, None, device)
    return workspace, p, workspace.numel() * workspace.element_size()


def gscan_workspace_size(x, layout="bct"):
    """Bytes of workspace gscan_fwd and gscan_bwd need for activations like x."""
    B, C, T = _rows_and_run(x.shape, layout)
    return _sizes(B, C, T, LAYOUTS[layout], _dtype_code(x))[1]


def gscan_fwd(x, r, i, lam, h0=None, lengths=None, layout="bct", reverse=False, decay=8.0, h=None,
              save_states=False, workspace=None, stream=None):
    """(h, h_last, states) of the recurrence: h like x, h_last [B, C] fp32 the state after the
    last valid position, states what gscan_bwd needs (None unless ``save_states``).  lam [C] and
    h0 [B, C] are fp32, lengths [B] int32 (see include/gscan.h)."""
    code, dt, dev = _input(x)
    s = _shape(x, code, layout, reverse, decay)
    shape, rows = x.shape, (s.B, s.C)
    px, pr, pi = _act("x", x, shape, dt, dev), _act("r", r, shape, dt, dev), _act("i", i, shape, dt, dev)
    plam = _flat("lam", lam, (s.C,), _f32, dev)
    ph0 = _flat("h0", h0, rows, _f32, dev)
    plen = _flat("lengths", lengths, (s.B,), _i32, dev)
    if h is not None:
        _act("h", h, shape, dt, dev)
    _on_gpu(dev)
    if h is None:
        h = torch.empty(shape, dtype=dt, device=dev)
    h_last = torch.empty(rows, dtype=_f32, device=dev)
    states = pstates = None
    if save_states:
        states = torch.empty(_sizes(s.B, s.C, s.T, s.layout, code)[0], dtype=_f32, device=dev)
        pstates = states.data_ptr()
    ws, pws, nws = _workspace(s, dev, workspace)
    _lib._check(_lib.lib.gscan_fwd(ctypes.byref(s), px, pr, pi, plam, ph0, plen,
                                   _act("h", h, shape, dt, dev), h_last.data_ptr(), pstates, pws, nws,
                                   _raw_stream(stream, dev)), "gscan_fwd")
    return h, h_last, states


def gscan_bwd(x, r, i, lam, states, dh, dh_last=None, lengths=None, layout="bct", reverse=False,
              decay=8.0, grads=None, workspace=None, stream=None):
    """Gradients of <dh, h> + <dh_last, h_last> as a dict keyed by GRAD_NAMES, from the inputs
    and the states of gscan_fwd.  ``grads`` may hold tensors to write (dx, dr, di with free
    strides); those it lacks are allocated."""
    grads = dict(grads or {})
    unknown = [n for n in grads if n not in GRAD_NAMES]
    if unknown:
        raise KeyError("unknown gradients %s" % ", ".join(map(str, unknown)))
    code, dt, dev = _input(x)
    s = _shape(x, code, layout, reverse, decay)
    shape, rows = x.shape, (s.B, s.C)
    px, pr, pi = _act("x", x, shape, dt, dev), _act("r", r, shape, dt, dev), _act("i", i, shape, dt, dev)
    pdh = _act("dh", dh, shape, dt, dev)
    plam = _flat("lam", lam, (s.C,), _f32, dev)
    plast = _flat("dh_last", dh_last, rows, _f32, dev)
    plen = _flat("lengths", lengths, (s.B,), _i32, dev)
    for n in ("dx", "dr", "di"):
        if grads.get(n) is not None:
            _act("grads[%s]" % n, grads[n], shape, dt, dev)
    for n, sh in (("dlam", (s.C,)), ("dh0", rows)):
        _flat("grads[%s]" % n, grads.get(n), sh, _f32, dev)
    if states is None:
        raise ValueError("gscan_bwd needs the states of gscan_fwd(..., save_states=True)")
    pst = _flat("states", states, (_sizes(s.B, s.C, s.T, s.layout, code)[0],), _f32, dev)
    _on_gpu(dev)
    for n in ("dx", "dr", "di"):
        if grads.get(n) is None:
            grads[n] = torch.empty(shape, dtype=dt, device=dev)
    for n, sh in (("dlam", (s.C,)), ("dh0", rows)):
        if grads.get(n) is None:
            grads[n] = torch.empty(sh, dtype=_f32, device=dev)
    ws, pws, nws = _workspace(s, dev, workspace)
    _lib._check(_lib.lib.gscan_bwd(ctypes.byref(s), px, pr, pi, plam, pst, plen, pdh, plast,
                                   *[_act(n, grads[n], shape, dt, dev) for n in ("dx", "dr", "di")],
                                   grads["dlam"].data_ptr(), grads["dh0"].data_ptr(), pws, nws,
                                   _raw_stream(stream, dev)), "gscan_bwd")
    return grads


def gscan_step(x, r, i, lam, state, slots=None, decay=8.0, h=None, stream=None):
    """One position of B sequences: x, r, i [B, C] (free row strides), their states in rows
    ``slots`` (int32 [B]; the first B rows if None) of ``state`` [S, C] fp32, which is updated.
    Returns h [B, C].  Sequences whose slot is outside 0..S-1 give zeros and change nothing."""
    code, dt, dev = _input(x)
    shape = x.shape
    if len(shape) != 2:
        raise ValueError("activations must be [B, C], got shape %s" % (tuple(shape),))
    B, C = shape
    px, pr, pi = _act("x", x, shape, dt, dev), _act("r", r, shape, dt, dev), _act("i", i, shape, dt, dev)
    plam = _flat("lam", lam, (C,), _f32, dev)
    pstate = _flat("state", state, None, _f32, dev)
    if state.dim() != 2 or state.shape[1] != C:
        raise ValueError("state must be [S, %d], got shape %s" % (C, tuple(state.shape)))
    S = state.shape[0]
    pslots = _flat("slots", slots, (B,), _i32, dev)
    if slots is None and S < B:
        raise ValueError("state has %d rows for %d sequences" % (S, B))
    _on_gpu(dev)
    if h is None:
        h = torch.empty(shape, dtype=dt, device=dev)
    _lib._check(_lib.lib.gscan_step(B, C, S, code, decay, px, pr, pi, plam, pstate, pslots,
                                    _act("h", h, shape, dt, dev), _raw_stream(stream, dev)),
                "gscan_step")
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
