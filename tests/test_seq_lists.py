"""Lists of tensors that the bindings of the AdamW step and of the recurrence
read: how long their tensors live, and tensors without memory.  CPU only."""
import weakref

import pytest
import torch

from aware_conv_amd import _lib as L
from aware_conv_amd import adamw, gscan


class Recorder:
    """Stands in for the library: notes which tensors are alive when the step is enqueued."""

    def __init__(self):
        self.seen, self.alive = [], None

    def column(self, ts, *_):
        assert isinstance(ts, (list, tuple))
        self.seen += [weakref.ref(t) for t in ts]
        return 0, len(ts)

    def written(self, *_):
        pass

    def enqueue(self, *_):
        self.alive = [r() is not None for r in self.seen]
        return 0


@pytest.mark.parametrize("name", ["grads", "exp_avgs", "exp_avg_sqs", "masters", "scales"])
def test_tensors_of_any_iterable_live_until_the_step_is_enqueued(monkeypatch, name):
    rec = Recorder()
    monkeypatch.setattr(adamw, "_lists", rec)
    monkeypatch.setattr(adamw, "_gpu_of", lambda _, ts: ts[0].device)
    monkeypatch.setattr(adamw, "_raw_stream", lambda *_: 0)
    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: None)  # that of CPU tensors

    class Lib:
        adamw_step = rec.enqueue
        adamw_workspace_size = L.lib.adamw_workspace_size

    monkeypatch.setattr(L, "lib", Lib)
    p = [torch.zeros(4), torch.zeros(4)]
    kw = {n: [torch.zeros(4), torch.zeros(4)] for n in ("grads", "exp_avgs", "exp_avg_sqs", "masters")}
    kw["scales"] = ([torch.zeros(1), torch.zeros(1)], [torch.zeros(1), torch.zeros(1)])
    temporary = lambda: (torch.zeros(4) for _ in range(2))  # noqa: E731
    kw[name] = (temporary(), temporary()) if name == "scales" else temporary()
    adamw.adamw_step(p, step=torch.zeros(1, dtype=torch.int32), **kw)
    assert len(rec.alive) == 14 and all(rec.alive)


def test_the_extension_takes_no_iterator():
    t = adamw._new_table(1)
    for ts in ((x for x in [torch.zeros(3)]), {0: torch.zeros(3)}, torch.zeros(1, 3), "a", None):
        with pytest.raises(TypeError, match="list or tuple"):
            gscan._lists.column(ts, t.ctypes.data, 1, 0, torch.float32, 0, 0)


def test_written_tensors_have_new_versions():
    a, b, c, d = (torch.zeros(2) for _ in range(4))
    with torch.inference_mode():
        e = torch.zeros(2)
    gscan._lists.written(a, None, [b, c], (), (d, e), e)
    assert [t._version for t in (a, b, c, d)] == [1, 1, 1, 1]
