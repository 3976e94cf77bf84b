"""Refusals of the token operators' entry points (selective scan, causal convolution, norm), before
any device call, and the tests' own fp64 reference.  CPU only: every call to the library here
fails validation, or has nothing to do."""
import copy
import ctypes
import os
import subprocess
import sys

import pytest
import torch

import token_reference as ref
from aware_conv_amd import _lib as L
from aware_conv_amd import SelectiveMixer, _acts, cconv, rmsnorm, sscan

NULL, SHAPE, DTYPE, ALIGN, WORKSPACE, UNSUPPORTED, ALIAS, LAYOUT, VALUE = -1, -2, -5, -6, -7, -8, -9, -11, -12


def far(i):
    """Distinct fake buffers 1 TiB apart, never dereferenced."""
    return (i + 1) << 40


def by_ref(v):
    return None if v is None else ctypes.byref(v) if isinstance(v, ctypes.Structure) else v


# the selective scan ------------------------------------------------------------

def sshape(**kw):
    return L.SscanShape(**{**dict(B=2, T=40, D=12, N=4, G=3, dtype=0), **kw})


def wide(i, s=None, **kw):
    s = s or sshape()
    return L.GscanView(**{**dict(p=far(i), sb=s.T * s.D, sr=s.D), **kw})


def low(i, s=None, **kw):
    s = s or sshape()
    return L.GscanView(**{**dict(p=far(i), sb=s.T * s.G * s.N, sr=s.G * s.N), **kw})


def sfwd(s=None, ws=far(40), nws=None, **kw):
    """No output's memory is there unless told otherwise: nothing may run."""
    s = s or sshape()
    a = dict(x=wide(0, s), dt=wide(1, s), a_log=far(2), b=low(3, s), c=low(4, s), d=far(5), z=wide(6, s),
             dt_bias=far(7), h0=far(8), lengths=far(9), y=wide(10, s, p=None), h_last=far(11), states=far(12))
    a.update(kw)
    return L.lib.sscan_fwd(ctypes.byref(s), *[by_ref(v) for v in a.values()], ws, nws or 0, None)


def sbwd(s=None, ws=far(40), nws=0, **kw):
    """Workspace too short unless told otherwise: nothing may run."""
    s = s or sshape()
    a = dict(x=wide(0, s), dt=wide(1, s), a_log=far(2), b=low(3, s), c=low(4, s), d=far(5), z=wide(6, s),
             dt_bias=far(7), states=far(12), lengths=far(9), dy=wide(13, s), dh_last=far(14), dx=wide(15, s),
             ddt=wide(16, s), da_log=far(17), db=low(18, s), dc=low(19, s), dd=far(20), dz=wide(21, s),
             ddt_bias=far(22), dh0=far(23))
    a.update(kw)
    return L.lib.sscan_bwd(ctypes.byref(s), *[by_ref(v) for v in a.values()], ws, nws, None)


SHAPES = [(dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(D=-1), SHAPE), (dict(T=(1 << 30) + 1), SHAPE),
          (dict(N=0), SHAPE), (dict(N=65), SHAPE), (dict(G=0), SHAPE), (dict(G=5), SHAPE), (dict(dtype=3), DTYPE),
          (dict(B=1 << 20, D=64, G=1), SHAPE), (dict(D=1 << 25, N=2, G=1, B=1), SHAPE),
          (dict(D=1 << 20, G=1 << 20, N=2, B=1), SHAPE),
          (dict(B=1 << 20, D=1, G=1), UNSUPPORTED), (dict(B=1 << 12, D=1, G=1, T=1 << 30), UNSUPPORTED)]


@pytest.mark.parametrize("call", [sfwd, sbwd])
@pytest.mark.parametrize("kw,code", SHAPES)
def test_scan_shapes(call, kw, code):
    assert call(sshape(**kw)) == code


def test_scan_forward_arguments():
    assert sfwd() == NULL  # y has no memory: everything before it is in order
    y = wide(10)
    for n in ("x", "dt", "a_log", "b", "c"):
        assert sfwd(**{n: None, "y": y}) == NULL, n
    for n in ("x", "dt", "z"):
        assert sfwd(**{n: wide(0, p=far(0) + 2)}) == ALIGN, n
        assert sfwd(**{n: wide(0, sb=-1)}) == LAYOUT and sfwd(**{n: wide(0, sr=-1)}) == LAYOUT
    assert sfwd(b=low(3, p=far(3) + 1)) == ALIGN and sfwd(c=low(4, sr=-1)) == LAYOUT
    assert sfwd(a_log=far(2) + 2) == ALIGN
    assert sfwd(x=wide(0, sb=1 << 60)) == SHAPE
    # outputs that meet something
    for kw in (dict(y=wide(0)), dict(y=wide(6)), dict(y=low(3)), dict(h_last=far(8), y=y), dict(states=far(2), y=y),
               dict(h_last=far(12), y=y), dict(y=wide(10, p=far(9)))):
        assert sfwd(**kw) == ALIAS, kw
    assert sfwd(y=wide(10, sr=11)) == LAYOUT and sfwd(y=wide(10, sb=0)) == LAYOUT
    # nothing to do
    e = sshape(B=0)
    none = L.GscanView(None, 0, 0)
    assert sfwd(e, x=none, dt=none, b=none, c=none, z=none, y=none, h0=None, h_last=None, states=None, ws=None) == 0


def test_scan_strides():
    """Fifteen rows of a stride are within 32 bits; a single position's stride does not matter."""
    for n in ("x", "dt", "z"):
        assert sfwd(**{n: wide(0, sr=(1 << 26) + 1), "y": wide(10)}, ws=None) == UNSUPPORTED, n
    assert sfwd(b=low(3, sr=(1 << 26) + 1), y=wide(10), ws=None) == UNSUPPORTED
    assert sfwd(y=wide(10, sb=1 << 33, sr=(1 << 26) + 1), ws=None) == UNSUPPORTED
    assert sbwd(dx=wide(15, sb=1 << 33, sr=(1 << 26) + 1)) == UNSUPPORTED and sbwd(dx=wide(15, sb=1 << 33, sr=1 << 26)) == WORKSPACE


def test_scan_workspace():
    s = sshape(T=4000)
    n = ctypes.c_size_t(0)
    assert L.lib.sscan_workspace_size(ctypes.byref(s), 0, ctypes.byref(n)) == 0 and n.value > 0
    y = wide(10, s)
    assert sfwd(s, y=y, nws=n.value - 1) == WORKSPACE and sfwd(s, y=y, ws=None, nws=n.value) == NULL
    assert sfwd(s, y=y, ws=far(40) + 4, nws=n.value) == ALIGN
    assert sfwd(s, y=y, ws=far(0), nws=n.value) == ALIAS
    m = ctypes.c_size_t(0)
    assert L.lib.sscan_workspace_size(ctypes.byref(s), 1, ctypes.byref(m)) == 0 and m.value > n.value
    assert L.lib.sscan_workspace_size(ctypes.byref(s), 1, None) == NULL
    assert L.lib.sscan_states_size(None, ctypes.byref(m)) == NULL


def test_scan_backward_arguments():
    assert sbwd() == WORKSPACE
    for n in ("x", "dt", "a_log", "b", "c", "states", "dy", "dx", "ddt", "da_log", "db", "dc", "dd", "dz",
              "ddt_bias", "d", "z", "dt_bias"):
        assert sbwd(**{n: None}) == NULL, n  # d, z and dt_bias come with their gradients, or not at all
    for kw in (dict(lengths=None), dict(dh_last=None), dict(dh0=None), dict(d=None, dd=None), dict(z=None, dz=None),
               dict(dt_bias=None, ddt_bias=None)):
        assert sbwd(**kw) == WORKSPACE, kw
    for kw in (dict(dx=wide(0)), dict(ddt=wide(15)), dict(dz=wide(13)), dict(db=low(3)), dict(dc=low(18)),
               dict(da_log=far(2)), dict(dd=far(22)), dict(dh0=far(12)), dict(ddt_bias=far(9))):
        assert sbwd(**kw) == ALIAS, kw
    # b's and c's gradients as parts of one buffer, z's beside x's
    s = sshape()
    part = lambda k: L.GscanView(far(18) + 4 * 12 * k, s.T * 30, 30)  # noqa: E731
    assert sbwd(db=part(0), dc=part(1)) == WORKSPACE and sbwd(db=part(1), dc=part(1)) == ALIAS


def sstep(S=5, s=None, **kw):
    s = s or sshape(T=1)
    a = dict(x=wide(0, s, sb=12), dt=wide(1, s, sb=12), a_log=far(2), b=low(3, s, sb=12), c=low(4, s, sb=12), d=far(5),
             z=wide(6, s, sb=12), dt_bias=far(7), state=far(8), slots=far(9), y=wide(10, s, p=None))
    a.update(kw)
    return L.lib.sscan_step(ctypes.byref(s), S, *[by_ref(v) for v in a.values()], None)


def test_scan_step_arguments():
    y = wide(10, sb=12)
    assert sstep() == NULL and sstep(S=-1) == SHAPE and sstep(S=1, slots=None) == SHAPE
    assert sstep(s=sshape(N=65)) == SHAPE and sstep(s=sshape(dtype=9)) == DTYPE
    for n in ("x", "dt", "a_log", "b", "c", "state"):
        assert sstep(**{n: None, "y": y}) == NULL, n
    for kw in (dict(y=wide(0, sb=12)), dict(state=far(2), y=y), dict(state=far(9), y=y)):
        assert sstep(**kw) == ALIAS, kw
    assert sstep(y=wide(10, sb=11)) == LAYOUT


# the causal convolution ------------------------------------------------------------

def cshape(**kw):
    return L.CconvShape(**{**dict(B=2, T=40, C=12, K=4, dtype=0, silu=1), **kw})


def cview(i, **kw):
    return L.GscanView(**{**dict(p=far(i), sb=480, sr=12), **kw})


def cfwd(s=None, **kw):
    a = dict(x=cview(0), w=far(1), bias=far(2), h0=far(3), lengths=far(4), y=cview(5, p=None), last=far(6))
    a.update(kw)
    return L.lib.cconv_fwd(ctypes.byref(s or cshape()), *[by_ref(v) for v in a.values()], None)


def cbwd(s=None, ws=far(20), nws=0, **kw):
    a = dict(x=cview(0), w=far(1), bias=far(2), h0=far(3), lengths=far(4), dy=cview(7), dlast=far(8), dx=cview(9),
             dw=far(10), dbias=far(11), dh0=far(12))
    a.update(kw)
    return L.lib.cconv_bwd(ctypes.byref(s or cshape()), *[by_ref(v) for v in a.values()], ws, nws, None)


@pytest.mark.parametrize("call", [cfwd, cbwd])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(C=-1), SHAPE), (dict(K=0), SHAPE), (dict(K=9), SHAPE),
    (dict(T=(1 << 30) + 1), SHAPE), (dict(dtype=-1), DTYPE), (dict(B=1 << 16, C=1 << 16), SHAPE),
    (dict(B=1, C=(1 << 25) + 1), SHAPE), (dict(B=8, T=1 << 30, C=129), UNSUPPORTED)])
def test_conv_shapes(call, kw, code):
    assert call(cshape(**kw)) == code


def test_conv_arguments():
    y = cview(5)
    assert cfwd() == NULL and cfwd(x=None, y=y) == NULL and cfwd(w=None, y=y) == NULL
    for kw in (dict(y=cview(0)), dict(last=far(0), y=y), dict(last=far(3), y=y), dict(y=cview(4)), dict(y=cview(6))):
        assert cfwd(**kw) == ALIAS, kw
    assert cfwd(y=cview(5, sr=11)) == LAYOUT and cfwd(x=cview(0, p=far(0) + 1)) == ALIGN
    assert cbwd() == WORKSPACE
    for n in ("x", "w", "dy", "dx", "dw", "bias", "dbias"):
        assert cbwd(**{n: None}) == NULL, n
    for kw in (dict(h0=None), dict(lengths=None), dict(dlast=None), dict(dh0=None), dict(bias=None, dbias=None)):
        assert cbwd(**kw) == WORKSPACE, kw
    for kw in (dict(dx=cview(7)), dict(dw=far(1)), dict(dbias=far(10)), dict(dh0=far(3))):
        assert cbwd(**kw) == ALIAS, kw
    n = ctypes.c_size_t(0)
    assert L.lib.cconv_workspace_size(ctypes.byref(cshape()), ctypes.byref(n)) == 0 and n.value > 0
    assert cbwd(ws=None, nws=n.value) == NULL and cbwd(ws=far(7), nws=n.value) == ALIAS
    s = cshape(T=1)
    step = lambda S=5, cache=far(3), slots=far(4), y=cview(5, p=None, sb=12): L.lib.cconv_step(  # noqa: E731
        ctypes.byref(s), S, by_ref(cview(0, sb=12)), far(1), far(2), cache, slots, by_ref(y), None)
    assert step() == NULL and step(S=-1) == SHAPE and step(S=1, slots=None) == SHAPE and step(cache=None) == NULL
    assert step(cache=far(1), y=cview(5, sb=12)) == ALIAS and step(y=cview(0, sb=12)) == ALIAS


# the norm --------------------------------------------------------------------------

def nshape(**kw):
    return L.RmsnormShape(**{**dict(B=2, T=5, C=12, dtype=0, rdtype=0, eps=1e-6), **kw})


def nview(i, **kw):
    return L.GscanView(**{**dict(p=far(i), sb=60, sr=12), **kw})


def nfwd(s=None, e4m3=False, **kw):
    a = dict(x=nview(0), residual=nview(1), w=far(2), y=nview(3, p=None), scale=far(6), total=nview(4), rstd=far(5))
    a.update(kw)
    if not e4m3:
        a.pop("scale")
    call = L.lib.rmsnorm_fwd_e4m3 if e4m3 else L.lib.rmsnorm_fwd
    return call(ctypes.byref(s or nshape()), *[by_ref(v) for v in a.values()], None)


def nbwd(s=None, ws=far(20), nws=0, **kw):
    a = dict(kept=nview(0), w=far(2), rstd=far(5), dy=nview(7), dtotal=nview(8), dx=nview(9), dresidual=nview(10),
             dw=far(11))
    a.update(kw)
    return L.lib.rmsnorm_bwd(ctypes.byref(s or nshape()), *[by_ref(v) for v in a.values()], ws, nws, None)


@pytest.mark.parametrize("call", [nfwd, nbwd])
@pytest.mark.parametrize("kw,code", [
    (dict(B=-1), SHAPE), (dict(T=-1), SHAPE), (dict(C=-1), SHAPE), (dict(C=(1 << 20) + 1), SHAPE),
    (dict(B=1 << 16, T=1 << 16), SHAPE), (dict(dtype=5), DTYPE), (dict(dtype=0, rdtype=2), DTYPE),
    (dict(dtype=1, rdtype=2), DTYPE), (dict(eps=-1.0), VALUE), (dict(eps=float("nan")), VALUE),
    (dict(eps=float("inf")), VALUE)])
def test_norm_shapes(call, kw, code):
    assert call(nshape(**kw)) == code


def test_norm_arguments():
    y = nview(3)
    for e in (False, True):
        assert nfwd(e4m3=e) == NULL and nfwd(e4m3=e, x=None, y=y) == NULL and nfwd(e4m3=e, w=None, y=y) == NULL
        # both or neither
        assert nfwd(e4m3=e, residual=None, y=y) == NULL and nfwd(e4m3=e, total=None, y=y) == NULL
        for kw in (dict(y=nview(0)), dict(y=nview(1)), dict(total=nview(0), y=y), dict(rstd=far(2), y=y),
                   dict(total=nview(1, p=far(1) + 4), y=y)):
            assert nfwd(e4m3=e, **kw) == ALIAS, kw
        # in place of the residual, and still not of x
        assert nfwd(e4m3=e, total=nview(1)) == NULL
        assert nfwd(e4m3=e, total=nview(0), residual=nview(0), y=y) == ALIAS
    assert nfwd(e4m3=True, scale=None, y=y) == NULL
    assert nfwd(y=nview(3, p=far(3) + 2)) == ALIGN and nfwd(y=nview(3, sr=11)) == LAYOUT
    assert nbwd() == WORKSPACE
    for n in ("kept", "w", "rstd", "dy"):
        assert nbwd(**{n: None}) == NULL, n
    for n in ("dtotal", "dx", "dresidual", "dw"):
        assert nbwd(**{n: None}) == WORKSPACE, n
    for kw in (dict(dx=nview(7)), dict(dresidual=nview(9)), dict(dw=far(2)), dict(dx=nview(8))):
        assert nbwd(**kw) == ALIAS, kw


# the bindings: the library sees only pointers and sizes ---------------------------------

def scan_args(**kw):
    z = torch.zeros
    return {**dict(x=z(2, 5, 6), dt=z(2, 5, 6), a_log=z(6, 4), b=z(2, 5, 8), c=z(2, 5, 8)), **kw}


@pytest.mark.parametrize("kw,error", [
    (dict(x=torch.zeros(2, 6)), ValueError), (dict(x=torch.zeros(2, 5, 6).double()), TypeError), (dict(x=None), TypeError),
    (dict(dt=torch.zeros(2, 5, 7)), ValueError), (dict(dt=torch.zeros(2, 5, 6).half()), TypeError),
    (dict(dt=None), TypeError), (dict(a_log=torch.zeros(7, 4)), ValueError), (dict(a_log=torch.zeros(6, 65)), ValueError),
    (dict(a_log=torch.zeros(6, 0)), ValueError), (dict(a_log=torch.zeros(6, 4).half()), TypeError),
    (dict(a_log=torch.zeros(4, 6).t()), ValueError),
    (dict(b=torch.zeros(2, 5, 6)), ValueError), (dict(b=torch.zeros(2, 5, 16)), ValueError),
    (dict(b=torch.zeros(2, 4, 8)), ValueError), (dict(b=torch.zeros(2, 5, 8).half()), TypeError),
    (dict(c=torch.zeros(2, 5, 4)), ValueError), (dict(c=None), TypeError), (dict(z=torch.zeros(2, 5, 5)), ValueError),
    (dict(z=torch.zeros(2, 6, 5).transpose(1, 2)), ValueError), (dict(d=torch.zeros(5)), ValueError),
    (dict(d=torch.zeros(6).half()), TypeError), (dict(dt_bias=torch.zeros(6, 1)), ValueError),
    (dict(lengths=torch.zeros(2)), TypeError), (dict(lengths=torch.zeros(3, dtype=torch.int32)), ValueError),
    (dict(h0=torch.zeros(2, 4, 6)), ValueError), (dict(y=torch.zeros(2, 5, 5)), ValueError),
    (dict(), ValueError)])  # everything in order, but not on a GPU
def test_scan_binding(kw, error):
    with pytest.raises(error):
        sscan.sscan_fwd(**scan_args(**kw))


def test_scan_backward_binding():
    a = scan_args()
    states, dy = torch.zeros(2 * 6 * 4), torch.zeros(2, 5, 6)
    for kw, error in ((dict(states=None), ValueError), (dict(states=torch.zeros(5)), ValueError),
                      (dict(dy=torch.zeros(2, 5, 5)), ValueError), (dict(dy=None), TypeError),
                      (dict(grads={"dq": dy}), KeyError), (dict(grads={"dz": dy}), ValueError),
                      (dict(grads={"dd": torch.zeros(6)}), ValueError), (dict(grads={"db": dy}), ValueError),
                      (dict(grads={"da_log": torch.zeros(4, 6)}), ValueError),
                      (dict(dh_last=torch.zeros(2, 6, 5)), ValueError), (dict(), ValueError)):
        with pytest.raises(error):
            sscan.sscan_bwd(*a.values(), **{**dict(states=states, dy=dy), **kw})


def test_scan_step_binding():
    z = torch.zeros
    a = dict(x=z(2, 6), dt=z(2, 6), a_log=z(6, 4), b=z(2, 8), c=z(2, 8), state=z(3, 6, 4))
    for kw, error in ((dict(state=z(1, 6, 4)), ValueError), (dict(state=z(3, 4, 6)), ValueError), (dict(state=None), TypeError),
                      (dict(x=z(2, 1, 6)), ValueError), (dict(slots=z(2)), TypeError), (dict(state=z(3, 6, 4).half()), TypeError),
                      (dict(), ValueError)):
        with pytest.raises(error):
            sscan.sscan_step(**{**a, **kw})


def test_conv_binding():
    z = torch.zeros
    a = dict(x=z(2, 5, 6), w=z(6, 4))
    for kw, error in ((dict(x=z(2, 6)), ValueError), (dict(w=z(6, 9)), ValueError), (dict(w=z(6, 0)), ValueError),
                      (dict(w=z(5, 4)), ValueError), (dict(w=z(6, 4).half()), TypeError), (dict(bias=z(5)), ValueError),
                      (dict(h0=z(2, 4, 6)), ValueError), (dict(h0=z(2, 3, 6).half()), TypeError),
                      (dict(lengths=z(2)), TypeError), (dict(y=z(2, 5, 6).half()), TypeError), (dict(), ValueError)):
        with pytest.raises(error):
            cconv.cconv_fwd(**{**a, **kw})
    for kw, error in ((dict(dy=z(2, 5, 5)), ValueError), (dict(dy=None), TypeError), (dict(grads={"dbias": z(6)}), ValueError),
                      (dict(grads={"q": z(6)}), KeyError), (dict(dlast=z(2, 2, 6)), ValueError), (dict(), ValueError)):
        with pytest.raises(error):
            cconv.cconv_bwd(**{**a, "dy": z(2, 5, 6), **kw})
    for kw, error in ((dict(cache=z(1, 3, 6)), ValueError), (dict(cache=z(3, 4, 6)), ValueError),
                      (dict(cache=z(3, 3, 6).half()), TypeError), (dict(), ValueError)):
        with pytest.raises(error):
            cconv.cconv_step(**{**dict(x=z(2, 6), w=z(6, 4), cache=z(3, 3, 6)), **kw})


def test_norm_binding():
    z = torch.zeros
    a = dict(x=z(2, 5, 6), w=z(6))
    for call in (rmsnorm.rmsnorm_fwd, rmsnorm.rmsnorm_fwd_e4m3):
        for kw, error in ((dict(x=z(6)), ValueError), (dict(w=z(5)), ValueError), (dict(w=z(6).half()), TypeError),
                          (dict(residual=z(2, 5, 5)), ValueError), (dict(residual=z(2, 5, 6).half()), TypeError),
                          (dict(total=z(2, 5, 6)), ValueError), (dict(x=z(2, 5, 6).half(), residual=z(2, 5, 6).bfloat16()), TypeError),
                          (dict(residual=z(2, 5, 6), total=z(2, 5, 6).half()), TypeError), (dict(), ValueError)):
            with pytest.raises(error):
                call(**{**a, **kw})
    b = dict(kept=z(2, 5, 6), w=z(6), rstd=z(2, 5), dy=z(2, 5, 6))
    for kw, error in ((dict(kept=z(2, 5, 5)), ValueError), (dict(kept=z(2, 5, 6).half()), TypeError), (dict(rstd=z(10)), ValueError),
                      (dict(dy=z(2, 5, 6).double()), TypeError), (dict(dtotal=z(2, 5, 6).half()), TypeError),
                      (dict(grads={"dresidual": z(2, 5, 6)}), ValueError), (dict(grads={"dw": z(5)}), ValueError),
                      (dict(), ValueError)):
        with pytest.raises(error):
            rmsnorm.rmsnorm_bwd(**{**b, **kw})


WRAPPED = """
import ctypes
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from aware_conv_amd import _acts, sscan

views = sscan._Views6()

def f(x):
    try:
        _acts._lists.read(ctypes.addressof(views), x, ((("x",), (x,)),), %(flats)s)
    except RuntimeError as e:
        print("raised", str(e).splitlines()[0], flush=True)
        raise KeyError("seen")

with FakeTensorMode():
    x = torch.empty(4, 3, 8, device="cuda")
    try:
        torch.vmap(f)(x)
    except KeyError:
        pass
"""


def test_wrapped_tensors_raise():
    """Tensors without memory of their own, as torch's transforms make them, are refused by an
    exception: in a process of its own, with fake tensors for those on a GPU."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    for flats in ("()", '(("x", x, torch.float32, (3, 8), False),)'):
        r = subprocess.run([sys.executable, "-c", WRAPPED % {"flats": flats}], capture_output=True, text=True, timeout=120,
                           cwd=root)
        assert r.returncode == 0 and r.stdout.startswith("raised"), r.stderr[-2000:]


def test_read_refuses_what_it_cannot_take():
    read, at = _acts._lists.read, ctypes.addressof(sscan._Views6())
    x = torch.zeros(2, 3)
    assert read(at, x, ((("x",), (x,)),), ()) is None  # not on a GPU
    assert read(at, 3, (), ()) is None
    for bad in ((at, x, [], ()), (at, x, (), None), ("a", x, (), ()), (at,)):
        with pytest.raises(TypeError):
            read(*bad)


# the reference -----------------------------------------------------------------------

def leaf(g, *n):
    return torch.randn(*n, generator=g, dtype=torch.float64).requires_grad_()


@pytest.mark.parametrize("lengths", [None, [7, 0, 3]])
def test_scan_reference_against_autograd(lengths):
    g = torch.Generator().manual_seed(0)
    B, T, D, N, G = 3, 7, 6, 3, 2
    p = {"x": leaf(g, B, T, D), "dt": leaf(g, B, T, D), "a_log": leaf(g, D, N), "b": leaf(g, B, T, G * N),
         "c": leaf(g, B, T, G * N), "d": leaf(g, D), "z": leaf(g, B, T, D), "dt_bias": leaf(g, D), "h0": leaf(g, B, D, N)}
    dy, dh = leaf(g, B, T, D).detach(), leaf(g, B, D, N).detach()
    loss = 0
    for i, n in enumerate(ref.counts(B, T, lengths)):
        h = p["h0"][i]
        for t in range(n):
            delta = torch.nn.functional.softplus(p["dt"][i, t] + p["dt_bias"])
            b, c = (p[k][i, t].view(G, 1, N).expand(G, D // G, N).reshape(D, N) for k in "bc")
            h = torch.exp(-delta[:, None] * torch.exp(p["a_log"])) * h + (delta * p["x"][i, t])[:, None] * b
            loss = loss + (dy[i, t] * ((c * h).sum(1) + p["d"] * p["x"][i, t]) * torch.nn.functional.silu(p["z"][i, t])).sum()
        loss = loss + (dh[i] * h).sum()
    loss.backward()
    out, mass = ref.sscan(lengths=lengths, dy=dy, dh_last=dh, **{k: t.detach() for k, t in p.items()})
    for k, t in p.items():
        assert torch.allclose(out["d" + k], t.grad, rtol=1e-10, atol=1e-12), k
    assert all((mass[k] >= out[k].abs() - 1e-12).all() for k in mass)


@pytest.mark.parametrize("lengths", [None, [7, 0, 2]])
@pytest.mark.parametrize("act", [True, False])
def test_conv_reference_against_autograd(lengths, act):
    g = torch.Generator().manual_seed(0)
    B, T, C, K = 3, 7, 5, 4
    p = {"x": leaf(g, B, T, C), "w": leaf(g, C, K), "bias": leaf(g, C), "h0": leaf(g, B, K - 1, C)}
    dy, dlast = leaf(g, B, T, C).detach(), leaf(g, B, K - 1, C).detach()
    loss = 0
    for i, n in enumerate(ref.counts(B, T, lengths)):
        line = torch.cat([p["h0"][i], p["x"][i, :n]])
        if n:
            v = torch.nn.functional.conv1d(line.t()[None], p["w"][:, None], p["bias"], groups=C)[0].t()
            loss = loss + (dy[i, :n] * (torch.nn.functional.silu(v) if act else v)).sum()
        loss = loss + (dlast[i] * line[n:]).sum()
    loss.backward()
    out, mass = ref.cconv(**{k: t.detach() for k, t in p.items()}, lengths=lengths, act=act, dy=dy, dlast=dlast)
    for k, n in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("h0", "dh0")):
        assert torch.allclose(out[n], p[k].grad, rtol=1e-10, atol=1e-12), k


def test_norm_reference_against_autograd():
    g = torch.Generator().manual_seed(0)
    x, w = leaf(g, 2, 3, 7), leaf(g, 7)
    dy, dt = leaf(g, 2, 3, 7).detach(), leaf(g, 2, 3, 7).detach()
    y = torch.nn.functional.rms_norm(x, (7,), w, 1e-3)
    ((y * dy).sum() + (x * dt).sum()).backward()
    out, _ = ref.rmsnorm(x.detach(), w.detach(), 1e-3, dy, dt)
    assert torch.allclose(out["y"], y.detach()) and torch.allclose(out["dx"], x.grad) and torch.allclose(out["dw"], w.grad)


def test_e4m3_reference():
    y = torch.linspace(-448, 448, 20001, dtype=torch.float64)
    assert torch.equal(ref.e4m3(y), y.float().to(torch.float8_e4m3fn).double())
    small = torch.linspace(-0.1, 0.1, 20001, dtype=torch.float64).float().double()
    assert torch.equal(ref.e4m3(small), small.float().to(torch.float8_e4m3fn).double())


# the block ---------------------------------------------------------------------------

@pytest.mark.parametrize("convert", [lambda m: m.half(), lambda m: m.to(torch.bfloat16), lambda m: copy.deepcopy(m).half()])
def test_block_conversions(convert):
    m = convert(SelectiveMixer(8, states=4))
    for n, p in m.named_parameters():
        assert p.dtype == (torch.float32 if n in m._FP32 else m.inner.weight.dtype), n
    assert m.inner.weight.dtype != torch.float32


def test_block_refuses_rows():
    m = SelectiveMixer(8, states=4)
    cache = m.new_cache(3)
    for rows in ([0], [0, 0], [0, 3], [-1, 0]):
        with pytest.raises(ValueError, match="rows must be"):
            m.prompt(torch.zeros(2, 5, 8), cache, rows=rows)
    with pytest.raises(TypeError):
        m.prompt(torch.zeros(2, 5, 8), cache, rows=[0.0, 1.0])
