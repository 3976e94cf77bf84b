"""The scan's states, 4 bytes per element of x with 16 states, are saved where a gradient may be asked
for, and only there.  CPU only: the library's call is replaced."""
import pytest
import torch

from aware_conv_amd import SelectiveMixer, cconv, rmsnorm, sscan


@pytest.fixture
def saved(monkeypatch):
    """What sscan_fwd was asked for, call by call."""
    asked = []

    def fwd(x, dt, a_log, b, c, save_states=False, **_):
        asked.append(save_states)
        return x * 1, x.new_zeros(x.shape[0], *a_log.shape), torch.zeros(4) if save_states else None

    monkeypatch.setattr(sscan, "sscan_fwd", fwd)
    return asked


def args(grad):
    x, b = torch.zeros(2, 5, 6), torch.zeros(2, 5, 4)
    return x, x + 1, torch.zeros(6, 4).requires_grad_(grad), b, b + 1


def test_states_are_saved_for_a_gradient(saved):
    y, _ = sscan.selective_scan(*args(True))
    assert saved == [True] and y.requires_grad


def test_the_function_applied_by_itself(saved, monkeypatch):
    """Without the last argument it keeps what a backward pass needs."""
    monkeypatch.setattr(sscan, "sscan_bwd", lambda *a, **k: {n: a[2] + 1 for n in sscan.GRAD_NAMES})
    a = args(True)
    y, _ = sscan.SelectiveScanFunction.apply(*a, *[None] * 5)
    y.sum().backward()
    assert saved == [True] and (a[2].grad == 1).all()


@pytest.mark.parametrize("mode", [torch.no_grad, torch.inference_mode])
def test_none_are_saved_without_one(saved, mode):
    sscan.selective_scan(*args(False))
    with mode():
        sscan.selective_scan(*args(True))
    assert saved == [False, False]


def test_none_are_saved_for_a_prompt(saved, monkeypatch):
    """The block's parameters require gradients; a prompt has none."""
    monkeypatch.setattr(rmsnorm, "rms_norm", lambda x, w, residual=None, eps=0: (x, None))
    monkeypatch.setattr(cconv, "causal_conv", lambda x, w, *a, **k: (x, x.new_zeros(len(x), w.shape[1] - 1, x.shape[2])))
    m = SelectiveMixer(8, states=4)
    x = torch.zeros(2, 5, 8)
    m.prompt(x, m.new_cache(3))
    assert saved == [False]
    m(x)
    assert saved == [False, True]
