"""Binding of the gated linear recurrence (include/gscan.h) and its autograd
function.

Activations are ``[B, C, T]`` (``layout="bct"``; also ``[B, C, H, W]`` planes,
taken in raster order) or ``[B, T, C]`` (``layout="btc"``), in float32, float16
or bfloat16.  Elements along the last axis are adjacent; the other strides are
free, so that x and the gates may be chunks of one projection.
"""
import ctypes

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
    n = t.dim()
    if t.numel() == 0:
        return True
    if n == 4:
        return ((t.shape[3] == 1 or t.stride(3) == 1) and
                (t.shape[2] == 1 or t.stride(2) == t.shape[3]))
    return t.shape[-1] == 1 or t.stride(-1) == 1


def _view(t):
    if t is None:
        return None
    return ctypes.byref(_lib.GscanView(t.data_ptr() or None, t.stride(0), t.stride(1)))


def _expect_acts(x, acts):
    for name, t in acts:
        if t is None:
            continue
        if not isinstance(t, torch.Tensor):
            raise TypeError("%s must be a torch.Tensor" % name)
        if t.shape != x.shape:
            raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(x.shape)))
        if t.dtype != x.dtype:
            raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, x.dtype))
        if not _adjacent(t):
            raise ValueError("%s must have adjacent elements along its rows" % name)


def _call(x, acts, flats, layout, reverse, decay, workspace):
    """Checks shared by fwd and bwd; `flats`: (name, tensor, shape, dtype).  Returns the shape
    struct."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    B, C, T = _rows_and_run(x.shape, layout)
    if T > MAX_T:
        raise ValueError("at most %d positions are supported, got %d" % (MAX_T, T))
    code = _dtype_code(x)
    _expect_acts(x, acts)
    for name, t, shape, dtype in flats:
        _lib._expect(dtype, [(name, t, shape(B, C))])
    _lib._expect(None, [("workspace", workspace, None)])
    _lib._on_gpu(x, list(acts) + [(n, t) for n, t, _, _ in flats] + [("workspace", workspace)])
    return _lib.GscanShape(B, C, T, LAYOUTS[layout], code, int(bool(reverse)), decay)


def _size(fn, s):
    n = ctypes.c_size_t(0)
    _lib._check(getattr(_lib.lib, fn)(ctypes.byref(s), ctypes.byref(n)), fn)
    return n.value


def _workspace(s, device, workspace):
    if workspace is None:
        need = _size("gscan_workspace_size", s)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=device)
    return workspace, workspace.numel() * workspace.element_size()


def _per_row(B, C):
    return (B, C)


def gscan_workspace_size(x, layout="bct"):
    """Bytes of workspace gscan_fwd and gscan_bwd need for activations like x."""
    B, C, T = _rows_and_run(x.shape, layout)
    return _size("gscan_workspace_size",
                 _lib.GscanShape(B, C, T, LAYOUTS[layout], _dtype_code(x), 0, 1.0))


def gscan_fwd(x, r, i, lam, h0=None, lengths=None, layout="bct", reverse=False, decay=8.0, h=None,
              save_states=False, workspace=None, stream=None):
    """(h, h_last, states) of the recurrence: h like x, h_last [B, C] fp32 the state after the
    last valid position, states what gscan_bwd needs (None unless ``save_states``).  lam [C] and
    h0 [B, C] are fp32, lengths [B] int32 (see include/gscan.h)."""
    s = _call(x, [("x", x), ("r", r), ("i", i), ("h", h)],
              [("lam", lam, lambda B, C: (C,), torch.float32), ("h0", h0, _per_row, torch.float32),
               ("lengths", lengths, lambda B, C: (B,), torch.int32)],
              layout, reverse, decay, workspace)
    dev = x.device
    if h is None:
        h = torch.empty(x.shape, dtype=x.dtype, device=dev)
    h_last = torch.empty((s.B, s.C), dtype=torch.float32, device=dev)
    states = None
    if save_states:
        states = torch.empty(_size("gscan_states_size", s) // 4, dtype=torch.float32, device=dev)
    ws, nws = _workspace(s, dev, workspace)
    p = _lib._ptr
    _lib._check(_lib.lib.gscan_fwd(ctypes.byref(s), _view(x), _view(r), _view(i), p(lam), p(h0),
                                   p(lengths), _view(h), p(h_last), p(states), p(ws), nws,
                                   _lib._stream(stream, dev)), "gscan_fwd")
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
    acts = [("x", x), ("r", r), ("i", i), ("dh", dh)]
    acts += [("grads[%s]" % n, grads.get(n)) for n in ("dx", "dr", "di")]
    flats = [("lam", lam, lambda B, C: (C,), torch.float32),
             ("dh_last", dh_last, _per_row, torch.float32),
             ("lengths", lengths, lambda B, C: (B,), torch.int32),
             ("grads[dlam]", grads.get("dlam"), lambda B, C: (C,), torch.float32),
             ("grads[dh0]", grads.get("dh0"), _per_row, torch.float32)]
    s = _call(x, acts, flats, layout, reverse, decay, workspace)
    if states is None:
        raise ValueError("gscan_bwd needs the states of gscan_fwd(..., save_states=True)")
    _lib._expect(torch.float32, [("states", states, (_size("gscan_states_size", s) // 4,))])
    _lib._on_gpu(x, [("states", states)])
    dev = x.device
    for n in ("dx", "dr", "di"):
        if grads.get(n) is None:
            grads[n] = torch.empty(x.shape, dtype=x.dtype, device=dev)
    for n, shape in (("dlam", (s.C,)), ("dh0", (s.B, s.C))):
        if grads.get(n) is None:
            grads[n] = torch.empty(shape, dtype=torch.float32, device=dev)
    ws, nws = _workspace(s, dev, workspace)
    p = _lib._ptr
    _lib._check(_lib.lib.gscan_bwd(ctypes.byref(s), _view(x), _view(r), _view(i), p(lam), p(states),
                                   p(lengths), _view(dh), p(dh_last),
                                   *[_view(grads[n]) for n in ("dx", "dr", "di")],
                                   p(grads["dlam"]), p(grads["dh0"]), p(ws), nws,
                                   _lib._stream(stream, dev)), "gscan_bwd")
    return grads


def gscan_step(x, r, i, lam, state, slots=None, decay=8.0, h=None, stream=None):
    """One position of B sequences: x, r, i [B, C] (free row strides), their states in rows
    ``slots`` (int32 [B]; the first B rows if None) of ``state`` [S, C] fp32, which is updated.
    Returns h [B, C].  Sequences whose slot is outside 0..S-1 give zeros and change nothing."""
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if x.dim() != 2:
        raise ValueError("activations must be [B, C], got shape %s" % (tuple(x.shape),))
    B, C = x.shape
    code = _dtype_code(x)
    acts = [("x", x), ("r", r), ("i", i), ("h", h)]
    _expect_acts(x, acts)
    if not isinstance(state, torch.Tensor):
        raise TypeError("state must be a torch.Tensor")
    if state.dim() != 2 or state.shape[1] != C:
        raise ValueError("state must be [S, %d], got shape %s" % (C, tuple(state.shape)))
    flats = [("lam", lam, (C,)), ("state", state, None)]
    _lib._expect(torch.float32, flats)
    _lib._expect(torch.int32, [("slots", slots, (B,))])
    if slots is None and state.shape[0] < B:
        raise ValueError("state has %d rows for %d sequences" % (state.shape[0], B))
    _lib._on_gpu(x, acts + [("lam", lam), ("state", state), ("slots", slots)])
    if h is None:
        h = torch.empty((B, C), dtype=x.dtype, device=x.device)
    p = _lib._ptr
    _lib._check(_lib.lib.gscan_step(B, C, state.shape[0], code, decay, _view(x), _view(r), _view(i),
                                    p(lam), p(state), p(slots), _view(h),
                                    _lib._stream(stream, x.device)), "gscan_step")
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
