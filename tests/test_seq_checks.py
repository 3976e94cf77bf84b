"""Refusals of the recurrence's and the AdamW step's entry points, before any
device call, and the tests' own fp64 reference.  CPU only: every call to the
library here fails validation."""
import ctypes

import numpy as np
import pytest
import torch

import seq_reference as ref
from aware_conv_amd import _lib as L
from aware_conv_amd import adamw, gscan

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, ALIAS, LAYOUT, VALUE = -1, -2, -5, -6, -7, -9, -11, -12


def far(i):
    """Distinct fake buffers 1 TiB apart, never dereferenced."""
    return (i + 1) << 40


def shape(**kw):
    d = dict(B=2, C=4, T=600, layout=0, dtype=0, reverse=0, decay=8.0)
    d.update(kw)
    return L.GscanShape(*(d[n] for n, _ in L.GscanShape._fields_))


def view(p, s=None, sb=None, sr=None):
    s = s or shape()
    rows, run = (s.C, s.T) if s.layout == 0 else (s.T, s.C)
    return L.GscanView(p, rows * run if sb is None else sb, run if sr is None else sr)


def fwd(s=None, ws=far(20), nws=0, **kw):
    """Workspace one byte short unless told otherwise: nothing may run."""
    s = s or shape()
    a = dict(x=view(far(0), s), r=view(far(1), s), i=view(far(2), s), lam=far(3), h0=far(4), lengths=far(5),
             h=view(far(6), s), h_last=far(7), states=far(8))
    a.update(kw)
    ref_ = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
    return L.lib.gscan_fwd(ctypes.byref(s), ref_(a["x"]), ref_(a["r"]), ref_(a["i"]), a["lam"], a["h0"],
                           a["lengths"], ref_(a["h"]), a["h_last"], a["states"], ws, nws, None)


def bwd(s=None, ws=far(20), nws=0, **kw):
    s = s or shape()
    a = dict(x=view(far(0), s), r=view(far(1), s), i=view(far(2), s), lam=far(3), states=far(4), lengths=far(5),
             dh=view(far(6), s), dh_last=far(7), dx=view(far(8), s), dr=view(far(9), s), di=view(far(10), s),
             dlam=far(11), dh0=far(12))
    a.update(kw)
    ref_ = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
    return L.lib.gscan_bwd(ctypes.byref(s), ref_(a["x"]), ref_(a["r"]), ref_(a["i"]), a["lam"], a["states"],
                           a["lengths"], ref_(a["dh"]), a["dh_last"], ref_(a["dx"]), ref_(a["dr"]),
                           ref_(a["di"]), a["dlam"], a["dh0"], ws, nws, None)


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), SHAPE), (dict(C=-1), SHAPE), (dict(T=-1), SHAPE), (dict(T=(1 << 30) + 1), SHAPE),
    (dict(B=1 << 15, C=1 << 15), SHAPE), (dict(dtype=3), DTYPE), (dict(dtype=-1), DTYPE),
    (dict(layout=2), LAYOUT), (dict(decay=0.0), VALUE), (dict(decay=-1.0), VALUE),
    (dict(decay=float("nan")), VALUE), (dict(decay=float("inf")), VALUE),
])
def test_shapes(call, kw, code):
    assert call(shape(**kw)) == code


@pytest.mark.parametrize("call", [fwd, bwd])
def test_launches_that_would_not_fit(call):
    assert call(shape(B=1 << 12, C=1, T=1 << 22, layout=1)) == -8
    assert call(shape(B=1 << 4, C=1 << 6, T=1 << 30)) == -8
    # the same tokens in whole tiles of channels
    assert call(shape(B=1 << 6, C=64, T=1 << 22, layout=1), ws=None) in (ALIAS, SHAPE, WORKSPACE)


def test_forward_arguments():
    assert fwd() == WORKSPACE  # everything before it is in order
    for n in ("x", "r", "i", "lam", "h"):
        assert fwd(**{n: None}) == NULL, n
    for n in ("h0", "lengths", "h_last", "states"):
        assert fwd(**{n: None}) == WORKSPACE, n
    for n in ("x", "r", "i", "h"):
        assert fwd(**{n: view(None)}) == NULL
        assert fwd(**{n: view(far(0) + 2)}) == ALIGN
        assert fwd(**{n: view(far(0), sb=-1)}) == LAYOUT
        assert fwd(**{n: view(far(0), sr=-4)}) == LAYOUT
    assert fwd(lam=far(3) + 1) == ALIGN
    # a length that would wrap
    assert fwd(x=view(far(0), sb=1 << 60)) == SHAPE
    # nothing to do: nothing is needed
    e = shape(B=0)
    assert fwd(e, x=view(None, e), r=view(None, e), i=view(None, e), h=view(None, e), ws=None) == 0


def test_outputs_may_not_meet_anything():
    for n, p in (("h", view(far(0))), ("h_last", far(0)), ("states", far(1)), ("h", view(far(3))),
                 ("h_last", far(4)), ("states", far(5)), ("h_last", far(6)), ("states", far(7))):
        assert fwd(**{n: p}) == ALIAS, (n, p)
    # the last element of x
    assert fwd(h_last=far(0) + 4 * (2 * 4 * 600 - 1)) == ALIAS
    # rows that overlap
    assert fwd(h=view(far(6), sr=599)) == LAYOUT
    assert fwd(h=view(far(6), sb=0)) == LAYOUT
    # inputs may be expanded
    assert fwd(r=view(far(1), sb=0, sr=0)) == WORKSPACE
    # a workspace over a buffer, where it is large enough to be used
    n = ctypes.c_size_t(0)
    assert L.lib.gscan_workspace_size(ctypes.byref(shape()), ctypes.byref(n)) == 0
    assert fwd(ws=far(0), nws=n.value + 64) == ALIAS
    assert fwd(ws=far(20) + 4, nws=n.value + 64) == ALIGN
    assert fwd(ws=None, nws=n.value + 64) == NULL


def test_backward_arguments():
    assert bwd() == WORKSPACE
    for n in ("x", "r", "i", "lam", "states", "dh", "dx", "dr", "di", "dlam"):
        assert bwd(**{n: None}) == NULL, n
    for n in ("lengths", "dh_last", "dh0"):
        assert bwd(**{n: None}) == WORKSPACE, n
    for n, p in (("dx", view(far(0))), ("dr", view(far(8))), ("di", view(far(6))), ("dlam", far(3)),
                 ("dh0", far(7)), ("dlam", far(4)), ("dh0", far(9))):
        assert bwd(**{n: p}) == ALIAS, n


@pytest.mark.parametrize("layout", [0, 1])
@pytest.mark.parametrize("B", [1, 2])
@pytest.mark.parametrize("C,T", [(4, 600), (4, 1), (1, 600), (1, 1)])
def test_parts_of_one_buffer(layout, B, C, T):
    """The chunks of a [B, 3C, T] or [B, T, 3C] tensor lie side by side; shifted by less they meet."""
    s = shape(B=B, C=C, T=T, layout=layout)
    run, rows = (T, C) if layout == 0 else (C, T)
    sr, sb = (T, 3 * C * T) if layout == 0 else (3 * C, 3 * C * T)
    step = C * T if layout == 0 else C
    parts = [view(far(8) + 4 * k * step, s, sb=sb, sr=sr) for k in range(3)]
    assert bwd(s, dx=parts[0], dr=parts[1], di=parts[2]) == WORKSPACE
    assert bwd(s, dx=parts[2], dr=parts[1], di=parts[0]) == WORKSPACE
    assert bwd(s, dx=parts[0], dr=parts[0]) == ALIAS
    if step > 1:
        assert bwd(s, dx=parts[0], dr=view(far(8) + 4 * (step - 1), s, sb=sb, sr=sr)) == ALIAS


def step(B=2, C=4, S=5, dtype=0, decay=8.0, **kw):
    a = dict(x=L.GscanView(far(0), C, 0), r=L.GscanView(far(1), C, 0), i=L.GscanView(far(2), C, 0), lam=far(3),
             state=far(4), slots=far(5), h=L.GscanView(far(6), C, 0))
    a.update(kw)
    ref_ = lambda v: ctypes.byref(v) if v is not None else None  # noqa: E731
    return L.lib.gscan_step(B, C, S, dtype, decay, ref_(a["x"]), ref_(a["r"]), ref_(a["i"]), a["lam"], a["state"],
                            a["slots"], ref_(a["h"]), None)


def test_step_arguments():
    assert step(B=-1) == SHAPE and step(S=-1) == SHAPE and step(dtype=7) == DTYPE and step(decay=0.0) == VALUE
    assert step(S=1, slots=None) == SHAPE  # rows 0..B-1 do not exist
    for n in ("x", "r", "i", "lam", "state", "h"):
        assert step(**{n: None}) == NULL, n
    assert step(h=L.GscanView(far(0), 4, 0)) == ALIAS
    assert step(h=L.GscanView(far(6), 3, 0)) == LAYOUT
    assert step(state=far(3)) == ALIAS and step(slots=far(4)) == ALIAS
    assert step(B=0) == 0


def table(**kw):
    t = np.zeros((2, 8), dtype=np.int64)
    for k in range(2):
        t[k] = [far(10 * k + j) for j in range(7)] + [1000]
    for n, v in kw.items():
        t[0, ["p", "g", "w", "m", "v", "ms", "vs", "n"].index(n)] = v or 0
    return t


def config(**kw):
    d = dict(dtype=0, bits=32, lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, weight_decay=0.0, grad_scale=1.0,
             max_norm=0.0, lr_dev=None, grad_scale_dev=None, norm=None)
    d.update(kw)
    return L.AdamwConfig(*(d[n] for n, _ in L.AdamwConfig._fields_))


def adam(t=None, count=2, step=far(60), ws=far(61), nws=0, **kw):
    t = table() if t is None else t
    c = config(**kw)
    return L.lib.adamw_step(ctypes.byref(c), t.ctypes.data, count, step, ws, nws, None)


def test_adamw_arguments():
    assert adam() == WORKSPACE
    assert adam(count=-1) == SHAPE and adam(table(n=-1)) == SHAPE and adam(table(n=(1 << 34) + 1)) == SHAPE
    assert adam(dtype=3) == DTYPE and adam(bits=16) == DTYPE
    for kw in (dict(lr=float("nan")), dict(beta1=1.0), dict(beta1=-0.1), dict(beta2=float("nan")), dict(eps=-1.0),
               dict(weight_decay=float("inf")), dict(grad_scale=float("nan")), dict(max_norm=-1.0)):
        assert adam(**kw) == VALUE, kw
    assert adam(max_norm=1.0) == NULL  # a norm is needed
    for n in ("p", "g", "m", "v", "w"):  # w: for all tensors or for none
        assert adam(table(**{n: None})) == NULL, n
    for n in ("ms", "vs"):
        assert adam(table(**{n: None}), bits=8) == NULL and adam(table(**{n: None})) == WORKSPACE
    for n in ("p", "g", "w", "m", "v"):
        assert adam(table(**{n: far(0) + 2})) == ALIGN, n
    assert adam(table(m=far(3) + 1), bits=8) == WORKSPACE  # codes are bytes
    assert adam(step=None) == NULL and adam(step=far(60) + 2) == ALIGN and adam(norm=far(9) + 1) == ALIGN
    assert adam(nws=64, ws=None) == NULL and adam(nws=64, ws=far(61) + 8) == ALIGN
    assert L.lib.adamw_step(None, table().ctypes.data, 2, far(60), far(61), 64, None) == NULL


def test_norm_arguments():
    def norm(dtype=0, t=table(), count=2, scale=1.0, out=far(50), ws=far(51), nws=0):
        return L.lib.adamw_grad_norm(dtype, t.ctypes.data, count, scale, None, out, ws, nws, None)
    assert norm() == WORKSPACE
    assert norm(dtype=9) == DTYPE and norm(count=-1) == SHAPE and norm(scale=float("inf")) == VALUE
    assert norm(t=table(g=None)) == NULL and norm(t=table(g=far(1) + 2)) == ALIGN
    assert norm(out=None) == NULL and norm(out=far(50) + 2) == ALIGN
    # 8192 elements to a partial sum
    n = ctypes.c_size_t(0)
    t = table(n=16385 * 8192)
    assert L.lib.adamw_workspace_size(t.ctypes.data, 2, ctypes.byref(n)) == 0 and n.value == 8 * 16386
    assert L.lib.adamw_workspace_size(t.ctypes.data, 2, None) == NULL


def test_binding_of_the_recurrence():
    x, lam = torch.zeros(2, 3, 8), torch.zeros(3)
    ok = dict(x=x, r=x, i=x, lam=lam)

    def call(fn=gscan.gscan_fwd, **kw):
        return fn(**dict(ok, **kw))

    with pytest.raises(ValueError, match="GPU"):
        call()
    with pytest.raises(ValueError, match="layout must be"):
        call(layout="cbt")
    with pytest.raises(ValueError, match=r"must be \[B, T, C\]"):
        call(x=torch.zeros(2, 3), layout="btc")
    with pytest.raises(ValueError, match=r"must be \[B, C, T\]"):
        call(x=torch.zeros(2))
    with pytest.raises(TypeError, match="float32, float16 and bfloat16"):
        call(x=x.double())
    with pytest.raises(ValueError, match="r has shape"):
        call(r=torch.zeros(2, 3, 7))
    with pytest.raises(TypeError, match="i has dtype"):
        call(i=x.half())
    with pytest.raises(ValueError, match="r must have adjacent elements"):
        call(r=torch.zeros(2, 8, 3).transpose(1, 2))
    with pytest.raises(ValueError, match="x must have adjacent elements"):
        call(x=torch.zeros(2, 3, 4, 8)[..., ::2], r=torch.zeros(2, 3, 4, 4), i=torch.zeros(2, 3, 4, 4))
    with pytest.raises(ValueError, match="lam has shape"):
        call(lam=torch.zeros(4))
    with pytest.raises(TypeError, match="lam has dtype"):
        call(lam=lam.half())
    with pytest.raises(ValueError, match="h0 has shape"):
        call(h0=torch.zeros(3, 2))
    with pytest.raises(TypeError, match="lengths has dtype"):
        call(lengths=torch.zeros(2))
    with pytest.raises(TypeError, match="x must be"):
        call(x=None)
    b = dict(fn=gscan.gscan_bwd, dh=x, states=torch.zeros(6))
    with pytest.raises(ValueError, match="GPU"):
        call(**b)
    with pytest.raises(ValueError, match="needs the states"):
        call(**dict(b, states=None))
    with pytest.raises(ValueError, match="states has shape"):
        call(**dict(b, states=torch.zeros(7)))
    with pytest.raises(KeyError, match="unknown gradients dy"):
        call(grads={"dy": x}, **b)
    with pytest.raises(ValueError, match=r"grads\[dr\] has shape"):
        call(grads={"dr": torch.zeros(1)}, **b)
    s = dict(fn=gscan.gscan_step, x=torch.zeros(2, 3), r=torch.zeros(2, 3), i=torch.zeros(2, 3), state=torch.zeros(4, 3))
    with pytest.raises(ValueError, match="GPU"):
        call(**s)
    with pytest.raises(ValueError, match="state must be"):
        call(**dict(s, state=torch.zeros(4, 2)))
    with pytest.raises(ValueError, match="state has 1 rows"):
        call(**dict(s, state=torch.zeros(1, 3)))
    with pytest.raises(TypeError, match="slots has dtype"):
        call(slots=torch.zeros(2, dtype=torch.int64), **s)


def test_binding_of_adamw():
    p = [torch.zeros(3)]
    step = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError, match="GPU"):
        adamw.adamw_step(p, p, p, p, step)
    with pytest.raises(ValueError, match="GPU"):
        adamw.adamw_grad_norm(p)
    with pytest.raises(ValueError, match="at least one"):
        adamw.adamw_grad_norm([])
    assert adamw.adamw_step([], [], [], [], step) is None
    w = [torch.nn.Parameter(torch.zeros(3))]
    for kw in (dict(bits=4), dict(betas=(0.9, 1.0)), dict(max_norm=0.0)):
        with pytest.raises(ValueError):
            adamw.AdamW(w, **kw)


def test_reference_gradients_against_differences():
    """The fp64 reference's gradients against central differences of its forward."""
    torch.manual_seed(0)
    B, C, T = 2, 2, 7
    a = {k: torch.randn(B, C, T, dtype=torch.float64) for k in ("x", "r", "i")}
    a["lam"] = torch.randn(C, dtype=torch.float64) - 2
    a["h0"] = torch.randn(B, C, dtype=torch.float64)
    dh, dl = torch.randn(B, C, T, dtype=torch.float64), torch.randn(B, C, dtype=torch.float64)
    for form in (dict(), dict(reverse=True, lengths=[7, 4]), dict(lengths=[0, 1])):
        def loss(b):
            h, last, _ = ref.fwd(b["x"], b["r"], b["i"], b["lam"], h0=b["h0"], **form)
            return float((h * dh).sum() + (last * dl).sum())
        g = ref.bwd(a["x"], a["r"], a["i"], a["lam"], dh, h0=a["h0"], dh_last=dl, **form)
        for n in ("x", "r", "i", "lam", "h0"):
            for k in range(a[n].numel()):
                b = {m: t.clone() for m, t in a.items()}
                b[n].view(-1)[k] += 1e-5
                up = loss(b)
                b[n].view(-1)[k] -= 2e-5
                # steps of 1e-5: 1e-10 of the third derivatives, 1e-11 of rounding
                assert abs((up - loss(b)) / 2e-5 - float(g["d" + n].reshape(-1)[k])) < 1e-8, (form, n, k)


def test_reference_codes_are_e4m3():
    codes = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn)
    assert torch.equal(codes.double(), torch.from_numpy(ref.CODE_VALUES))
