"""Binding of the selective state space scan (include/sscan.h) and its autograd function.

Activations are token sequences ``[B, T, D]`` (``b`` and ``c``: ``[B, T, G * N]``) in float32,
float16 or bfloat16.  Elements along the last axis are adjacent; the other strides are free, so
that they may be parts of projections.  Parameters and states are float32."""
import ctypes
import functools

import torch

from . import _acts, _lib, gscan
from ._acts import VIEW, f32, i32
from .gscan import _lists, _raw_stream, _view, on_stream

GRAD_NAMES = ("dx", "ddt", "da_log", "db", "dc", "dd", "dz", "ddt_bias", "dh0")
MAX_T = 1 << 30
MAX_STATES = 64
_Views6, _Views11 = _lib.GscanView * 6, _lib.GscanView * 11


@functools.lru_cache(maxsize=256)
def _form(*shape):
    """The shape as the library takes it; it is only read."""
    return ctypes.byref(_lib.SscanShape(*shape))


@functools.lru_cache(maxsize=256)
def _sizes(*shape):
    """(floats of the states, bytes of the forward's workspace, of the backward's) for a shape."""
    s, n = _lib.SscanShape(*shape), ctypes.c_size_t(0)
    ref, out = ctypes.byref(s), []
    _lib._check(_lib.lib.sscan_states_size(ref, ctypes.byref(n)), "sscan_states_size")
    out.append(n.value // 4)
    for backward in (0, 1):
        _lib._check(_lib.lib.sscan_workspace_size(ref, backward, ctypes.byref(n)), "sscan_workspace_size")
        out.append(n.value)
    return out


def _shape(x, a_log, b, axes):
    """(B, T, D, N, G, dtype code) from the tensors that the others go by."""
    what = "[B, T, D]" if axes == 3 else "[B, D]"
    code = gscan._dtype_code(_acts.tensor("x", x))
    size = _acts.dims("x", x, axes, what)
    B, T, D = size[0], (size[1] if axes == 3 else 1), size[-1]
    if T > MAX_T:
        raise ValueError("at most %d positions are supported, got %d" % (MAX_T, T))
    n = _acts.dims("a_log", a_log, 2, "[D, N]")
    if n[0] != D or not 1 <= n[1] <= MAX_STATES:
        raise ValueError("a_log has shape %s, expected [%d, N] with N of 1 to %d" % (tuple(n), D, MAX_STATES))
    N = n[1]
    low = _acts.dims("b", b, axes, what.replace("D", "G * N"))
    G = low[-1] // N
    if low[:-1] != size[:-1] or low[-1] % N or G < 1 or D % G:
        raise ValueError("b has shape %s, expected %s and G * %d with G a divisor of %d"
                         % (tuple(low), tuple(size[:-1]), N, D))
    _acts.same_type(x, (("b", b),))
    return B, T, D, N, G, code


def sscan_workspace_size(x, a_log, b, backward=False):
    """Bytes of workspace sscan_fwd (``backward``: sscan_bwd) needs for tensors like these."""
    return _sizes(*_shape(x, a_log, b, 3))[2 if backward else 1]


@on_stream
def sscan_fwd(x, dt, a_log, b, c, d=None, z=None, dt_bias=None, h0=None, lengths=None, y=None,
              save_states=False, workspace=None, *, stream=None):
    """(y, h_last, states): y like x, h_last [B, D, N] fp32 the state after the last valid
    position, states what sscan_bwd needs (None unless ``save_states``).  a_log [D, N], d [D],
    dt_bias [D] and h0 [B, D, N] are fp32, lengths [B] int32; d, z, dt_bias and h0 may be None
    (see include/sscan.h)."""
    shape = B, T, D, N, G, code = _shape(x, a_log, b, 3)
    v = _Views6()
    p, (pa, pd, pbias, ph0, plen) = _acts.read(
        v, x, ((("x", "dt", "z", "y"), (x, _acts.tensor("dt", dt), z, y)),
               (("b", "c"), (b, _acts.tensor("c", c)))),
        (("a_log", a_log, f32, (D, N), False), ("d", d, f32, (D,), True), ("dt_bias", dt_bias, f32, (D,), True),
         ("h0", h0, f32, (B, D, N), True), ("lengths", lengths, i32, (B,), True)))
    dev, given = x.device, y
    if y is None:
        y = _acts.like(x)
        v[3] = _view(y)
    h_last = torch.empty((B, D, N), dtype=f32, device=dev)
    n_states, need, _ = _sizes(*shape)
    states = torch.empty(n_states, dtype=f32, device=dev) if save_states else None
    ws, pws, nws = _acts.workspace(need, dev, workspace)
    _lib._enqueue(dev, "sscan_fwd", _form(*shape), p, p + VIEW, pa, p + 4 * VIEW,
                  p + 5 * VIEW, pd, None if z is None else p + 2 * VIEW, pbias, ph0, plen, p + 3 * VIEW,
                  h_last.data_ptr(), None if states is None else states.data_ptr(), pws, nws,
                  _raw_stream(stream, dev))
    if given is not None:
        _lists.written(given)
    return y, h_last, states


@on_stream
def sscan_bwd(x, dt, a_log, b, c, states, dy, d=None, z=None, dt_bias=None, dh_last=None, lengths=None,
              grads=None, workspace=None, *, stream=None):
    """Gradients of <dy, y> + <dh_last, h_last> as a dict keyed by GRAD_NAMES, from the inputs and
    the states of sscan_fwd; those of d, z and dt_bias are there where they are.  ``grads`` may hold
    tensors to write (dx, ddt, dz, db, dc with free strides); those it lacks are allocated."""
    given = tuple((grads or {}).values())
    grads = _acts.known(grads, GRAD_NAMES)
    shape = B, T, D, N, G, code = _shape(x, a_log, b, 3)
    for name, t in (("dd", d), ("dz", z), ("ddt_bias", dt_bias)):
        if t is None and grads.get(name) is not None:
            raise ValueError("grads[%s] is given without %s" % (name, name[1:]))
    if states is None:
        raise ValueError("sscan_bwd needs the states of sscan_fwd(..., save_states=True)")
    n_states, _, need = _sizes(*shape)
    v = _Views11()
    get = grads.get
    p, (pa, pd, pbias, pst, plen, plast, pda, pdd, pdbias, pdh0) = _acts.read(
        v, x, ((("x", "dt", "z", "dy", "grads[dx]", "grads[ddt]", "grads[dz]"),
                (x, _acts.tensor("dt", dt), z, _acts.tensor("dy", dy), get("dx"), get("ddt"), get("dz"))),
               (("b", "c", "grads[db]", "grads[dc]"), (b, _acts.tensor("c", c), get("db"), get("dc")))),
        (("a_log", a_log, f32, (D, N), False), ("d", d, f32, (D,), True), ("dt_bias", dt_bias, f32, (D,), True),
         ("states", states, f32, (n_states,), False), ("lengths", lengths, i32, (B,), True),
         ("dh_last", dh_last, f32, (B, D, N), True), ("grads[da_log]", get("da_log"), f32, (D, N), True),
         ("grads[dd]", get("dd"), f32, (D,), True), ("grads[ddt_bias]", get("ddt_bias"), f32, (D,), True),
         ("grads[dh0]", get("dh0"), f32, (B, D, N), True)))
    dev = x.device
    for k, n, like in ((4, "dx", x), (5, "ddt", x), (6, "dz", z), (9, "db", b), (10, "dc", b)):
        if get(n) is None and like is not None:
            grads[n] = _acts.like(like)
            v[k] = _view(grads[n])
    out = []
    for n, at, size, there in (("da_log", pda, (D, N), True), ("dd", pdd, (D,), d is not None),
                               ("ddt_bias", pdbias, (D,), dt_bias is not None), ("dh0", pdh0, (B, D, N), True)):
        if at is None and there:
            grads[n] = torch.empty(size, dtype=f32, device=dev)
            at = grads[n].data_ptr()
        out.append(at)
    ws, pws, nws = _acts.workspace(need, dev, workspace)
    _lib._enqueue(dev, "sscan_bwd", _form(*shape), p, p + VIEW, pa, p + 7 * VIEW,
                  p + 8 * VIEW, pd, None if z is None else p + 2 * VIEW, pbias, pst, plen, p + 3 * VIEW, plast,
                  p + 4 * VIEW, p + 5 * VIEW, out[0], p + 9 * VIEW, p + 10 * VIEW, out[1],
                  None if z is None else p + 6 * VIEW, out[2], out[3], pws, nws, _raw_stream(stream, dev))
    _lists.written(given)
    return {n: grads.get(n) for n in GRAD_NAMES}


@on_stream
def sscan_step(x, dt, a_log, b, c, state, d=None, z=None, dt_bias=None, slots=None, y=None, *, stream=None):
    """One position of B sequences: x, dt, z [B, D] and b, c [B, G * N] (free row strides), their
    states in rows ``slots`` (int32 [B]; the first B rows if None) of ``state`` [S, D, N] fp32,
    which is updated.  Returns y [B, D].  Sequences whose slot is outside 0..S-1 give zeros and
    change nothing."""
    shape = B, _, D, N, G, code = _shape(x, a_log, b, 2)
    S = _acts.dims("state", state, 3, "[S, D, N]")[0]
    if slots is None and S < B:
        raise ValueError("state has %d rows for %d sequences" % (S, B))
    v = _Views6()
    p, (pa, pd, pbias, pstate, pslots) = _acts.read(
        v, x, ((("x", "dt", "z", "y"), (x, _acts.tensor("dt", dt), z, y)),
               (("b", "c"), (b, _acts.tensor("c", c)))),
        (("a_log", a_log, f32, (D, N), False), ("d", d, f32, (D,), True), ("dt_bias", dt_bias, f32, (D,), True),
         ("state", state, f32, (S, D, N), False), ("slots", slots, i32, (B,), True)))
    dev, given = x.device, y
    if y is None:
        y = _acts.like(x)
        v[3] = _view(y)
    _lib._enqueue(dev, "sscan_step", _form(*shape), S, p, p + VIEW, pa, p + 4 * VIEW,
                  p + 5 * VIEW, pd, None if z is None else p + 2 * VIEW, pbias, pstate, pslots, p + 3 * VIEW,
                  _raw_stream(stream, dev))
    _lists.written(state, given)
    return y


class SelectiveScanFunction(torch.autograd.Function):
    """Forward through ``sscan_fwd``, backward through ``sscan_bwd``.  Saved are the inputs and the
    states that pieces of the sequence start from; the others are formed again by the backward
    kernel."""

    @staticmethod
    def forward(ctx, x, dt, a_log, b, c, d, z, dt_bias, h0, lengths, grad=True):
        ctx.set_materialize_grads(False)
        x, dt, b, c, z = (_acts.rows(t) for t in (x, dt, b, c, z))
        a_log, d, dt_bias, h0 = (_acts.flat(t) for t in (a_log, d, dt_bias, h0))
        # needs_input_grad says what the inputs are, also where no gradient is recorded (grad=False)
        want = grad and any(ctx.needs_input_grad[:9])
        y, h_last, states = sscan_fwd(x, dt, a_log, b, c, d=d, z=z, dt_bias=dt_bias, h0=h0, lengths=lengths,
                                      save_states=want)
        if want:
            ctx.save_for_backward(x, dt, a_log, b, c, d, z, dt_bias, lengths, states)
        return y, h_last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, dy, dh_last):
        x, dt, a_log, b, c, d, z, dt_bias, lengths, states = ctx.saved_tensors
        if dy is None:
            dy = torch.zeros(x.shape, dtype=x.dtype, device=x.device)
        g = sscan_bwd(x, dt, a_log, b, c, states, _acts.rows(dy), d=d, z=z, dt_bias=dt_bias,
                      dh_last=_acts.flat(dh_last), lengths=lengths)
        order = ("dx", "ddt", "da_log", "db", "dc", "dd", "dz", "ddt_bias", "dh0")
        return (*[g[n] if need else None for n, need in zip(order, ctx.needs_input_grad)], None, None)


def selective_scan(x, dt, a_log, b, c, d=None, z=None, dt_bias=None, h0=None, lengths=None):
    """(y, h_last) of the selective state space scan, differentiable in every argument but
    ``lengths``."""
    return SelectiveScanFunction.apply(x, dt, a_log, b, c, d, z, dt_bias, h0, lengths, torch.is_grad_enabled())
