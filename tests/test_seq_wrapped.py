"""Tensors that have no memory of their own, as torch's function transforms make
them, are refused by an exception.  CPU only, in a process of its own: tensors on
a GPU are stood in for by fake ones, which have no memory either."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

CODE = """
import ctypes
import torch
from torch._subclasses.fake_tensor import FakeTensorMode
from aware_conv_amd import adamw, gscan

views, table = gscan._Views4(), adamw._new_table(1)
calls = {
    "views": lambda x: gscan._lists.views((x,), ctypes.addressof(views)),
    "flat": lambda x: gscan._lists.flat(x, torch.float32, 0, 3, 8),
    "column": lambda x: gscan._lists.column([x], table.ctypes.data, 1, 0, torch.float32, 0, 0),
}
call = calls[%(call)r]

def f(x):
    try:
        call(x)
    except RuntimeError as e:
        print("raised", str(e).splitlines()[0], flush=True)
        raise KeyError("seen")  # the transform itself has nothing to run on here

with FakeTensorMode():
    x = torch.empty(4, 3, 8, device="cuda")
    try:
        if %(transform)r == "vmap":
            torch.vmap(f)(x)
        else:
            torch.func.grad(f)(x[0])
    except KeyError:
        pass
"""


@pytest.mark.parametrize("transform", ["vmap", "grad"])
@pytest.mark.parametrize("call", ["views", "flat", "column"])
def test_wrapped_tensors_raise(call, transform):
    r = subprocess.run([sys.executable, "-c", CODE % {"call": call, "transform": transform}], capture_output=True,
                       text=True, timeout=120, cwd=ROOT)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.startswith("raised"), r.stdout
