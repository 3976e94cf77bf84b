"""The example's block of WTConv layers and recurrences, trained with AdamW:
the operators together, as a user has them."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
pytestmark = pytest.mark.gpu


def example():
    spec = importlib.util.spec_from_file_location("train_mixer", os.path.join(ROOT, "examples", "train_mixer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


@pytest.mark.parametrize("bits,dtype", [(32, torch.float32), (8, torch.float32), (8, torch.float16)])
def test_training_learns(bits, dtype):
    print("\ncase mixer %s %s" % (bits, dtype), flush=True)
    losses, block = example().train(steps=60, bits=bits, dtype=dtype)
    assert torch.isfinite(losses).all()
    # the target's mean is 1 and the untrained output's far from it: half is far less than it learns
    assert losses[-5:].mean() < 0.5 * losses[:3].mean()
    assert all(p.grad is not None and torch.isfinite(p.grad).all() for p in block.parameters())


def test_two_runs_agree_bit_for_bit():
    m = example()
    a, b = m.train(steps=5)[0], m.train(steps=5)[0]
    assert torch.equal(a, b)


def test_serving_agrees_with_one_pass():
    m = example()
    block = m.Block(16, device="cuda")
    # states of size 1 formed by the same formula in two groupings: 1e-5
    assert m.serve(block) <= 1e-5


def test_both_directions():
    """GatedScan2d against its parts."""
    import aware_conv_amd as A
    torch.manual_seed(0)
    layer = A.GatedScan2d(6, kernel_size=3, levels=2, device="cuda")
    x = torch.randn(2, 6, 12, 16, device="cuda")
    r, i = layer.reset(x), layer.input(x)
    f = A.gated_scan(x, r, i, layer.lam[0])[0]
    b = A.gated_scan(x.flatten(2).flip(2), r.flatten(2).flip(2), i.flatten(2).flip(2), layer.lam[1])[0]
    want = (f + b.flip(2).view_as(f)) / 2 ** 0.5
    # the same elements in other groupings of a tile: 1e-5 of the largest
    assert (layer(x) - want).abs().max() <= 1e-5 * want.abs().max()
