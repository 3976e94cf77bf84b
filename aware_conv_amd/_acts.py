"""Checks of what the token operators (sscan.py, cconv.py, rmsnorm.py) are given, and what the
library takes of it.

Tensors are checked and read by a small extension (pyext/tensor_lists.cpp); what it refuses is
looked at again here, to say what is wrong."""
import ctypes

import torch

from . import _lib, gscan
from .gscan import _lists

f32, i32 = torch.float32, torch.int32
VIEW = ctypes.sizeof(_lib.GscanView)


def tensor(name, t):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    return t


def dims(name, t, n, what):
    """The shape of `t`, which must have n axes."""
    if tensor(name, t).dim() != n:
        raise ValueError("%s must be %s, got shape %s" % (name, what, tuple(t.shape)))
    return t.shape


def same_type(x, tensors):
    """A reading as views leaves the first of a group to the caller: its type and device are x's."""
    for name, t in tensors:
        if tensor(name, t).dtype is not x.dtype:
            raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, x.dtype))


def read(out, x, groups, flats):
    """Writes the views of the activations into `out` and returns (its address, the addresses of
    `flats`).

    groups: (names, tensors); the tensors of a group are of one shape and dtype, the first's, and
    the others may be None.  flats: (name, tensor, dtype, dims, optional), contiguous.  All are on
    x's device."""
    at = ctypes.addressof(out)
    ps = _lists.read(at, x, groups, flats)
    if ps is None:
        _refuse(x, groups, flats)
    return at, ps


def _refuse(x, groups, flats):
    """Raises what is wrong: shapes first, devices last."""
    for names, tensors in groups:
        like = tensors[0]
        for name, t in zip(names, tensors):
            if t is None:
                continue
            tensor(name, t)
            if t.shape != like.shape:
                raise ValueError("%s has shape %s, expected %s" % (name, tuple(t.shape), tuple(like.shape)))
            if t.dtype is not like.dtype:
                raise TypeError("%s has dtype %s, expected %s" % (name, t.dtype, like.dtype))
            if not gscan._adjacent(t):
                raise ValueError("%s must have adjacent elements along its rows" % name)
    for name, t, dtype, n, optional in flats:
        if t is None and not optional:
            raise TypeError("%s must be a torch.Tensor" % name)
        _lib._expect(dtype, [(name, t, n)])
    _lib._on_gpu(x, [p for names, tensors in groups for p in zip(names, tensors)] + [f[:2] for f in flats])
    raise ValueError("tensors of an unsupported kind")


def rows(t):
    """`t` with adjacent elements along its last axis."""
    return t if t is None or gscan._adjacent(t) else t.contiguous()


def flat(t):
    return None if t is None else t.contiguous()


def workspace(need, device, given):
    """(tensor, address, bytes); the caller keeps the tensor until the call was enqueued."""
    if given is None:
        if need == 0:
            return None, None, 0
        given = torch.empty(need, dtype=torch.uint8, device=device)
    elif not given.is_contiguous():
        raise ValueError("workspace must be contiguous")
    elif given.device != device:
        raise ValueError("workspace is on %s; every tensor must be on %s" % (given.device, device))
    return given, given.data_ptr(), given.numel() * given.element_size()


def like(t):
    """An output like `t`, contiguous (half the time of torch.empty with its shape, dtype and device)."""
    return torch.empty_like(t, memory_format=torch.contiguous_format)


def known(grads, names):
    """A copy of the tensors to write, by name."""
    unknown = [n for n in grads or {} if n not in names]
    if unknown:
        raise KeyError("unknown gradients %s" % ", ".join(map(str, unknown)))
    return dict(grads or {})
