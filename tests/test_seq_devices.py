"""Calls whose tensors are on a device that is not the current one.  CPU only: the devices are
stood in for, and the library is not called."""
import types

import pytest
import torch

from aware_conv_amd import _lib as L
from aware_conv_amd import gscan


class Devices:
    """Device 0 is current, unless a context makes another one so."""

    def __init__(self):
        self.current, self.calls = 0, []

    def device(self, d):
        class Context:
            def __enter__(_):
                _.before, self.current = self.current, torch.device(d).index

            def __exit__(_, *e):
                self.current = _.before

        return Context()

    def __getattr__(self, name):  # the library: notes what was current
        def call(*args):
            self.calls.append((name, self.current, args))
            return 0
        return call


@pytest.fixture
def devices(monkeypatch):
    d = Devices()
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: d.current)
    monkeypatch.setattr(torch.cuda, "device", d.device)
    monkeypatch.setattr(L, "lib", d)
    return d


def test_the_library_is_called_with_the_tensors_device_current(devices):
    for k in (0, 1, 3):
        L._enqueue(torch.device("cuda", k), "gscan_step", "a", k)
        assert devices.calls.pop() == ("gscan_step", k, ("a", k)) and devices.current == 0


def test_errors_leave_the_device_as_it_was(devices, monkeypatch):
    monkeypatch.setattr(L, "lib", types.SimpleNamespace(gscan_fwd=lambda: -9, wtconv_strerror=lambda c: b""))
    with pytest.raises(L.WTConvError):
        L._enqueue(torch.device("cuda", 1), "gscan_fwd")
    assert devices.current == 0


def test_a_stream_of_another_device_is_refused():
    s = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=77)
    assert gscan._raw_stream(s, torch.device("cuda", 0)) == 77
    with pytest.raises(ValueError, match="stream is on cuda:0"):
        gscan._raw_stream(s, torch.device("cuda", 1))


def test_every_entry_point_goes_that_way():
    """No call enqueues through the library's handle itself."""
    import inspect
    from aware_conv_amd import adamw
    for module in (L, gscan, adamw):
        for line in inspect.getsource(module).splitlines():
            for name in L.EXPORTED:
                if not name.endswith(("_size", "strerror")) and ".argtypes" not in line and ".restype" not in line:
                    assert "lib.%s(" % name not in line, line
