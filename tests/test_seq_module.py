"""GatedScan2d under the conversions that a user applies to a whole model.  CPU only."""
import copy

import pytest
import torch

from aware_conv_amd import GatedScan2d


@pytest.mark.parametrize("convert", [lambda m: m.half(), lambda m: m.to(torch.bfloat16), lambda m: m.to(dtype=torch.float16),
                                     lambda m: m.type(torch.float16), lambda m: m.bfloat16().float()])
@pytest.mark.parametrize("inside", [False, True])
def test_lam_stays_as_it_is(convert, inside):
    """lam, its gradient and its identity, whatever the layer's dtype becomes."""
    layer = GatedScan2d(5, kernel_size=3, levels=1)
    lam, was = layer.lam, layer.lam.detach().clone()
    lam.grad = torch.rand_like(lam)
    grad = lam.grad.clone()
    convert(torch.nn.Sequential(layer) if inside else layer)
    assert layer.lam is lam and lam.dtype == torch.float32 and torch.equal(lam, was)
    assert lam.grad.dtype == torch.float32 and torch.equal(lam.grad, grad)
    want = torch.float32 if layer.reset.w_base.dtype == torch.float32 else layer.reset.w_base.dtype
    assert all(p.dtype == want for n, p in layer.named_parameters() if n != "lam")


def test_other_conversions():
    layer = GatedScan2d(5, kernel_size=3, levels=1).half()
    other = GatedScan2d(5, kernel_size=3, levels=1, dtype=torch.float16)
    other.load_state_dict(layer.state_dict())
    assert torch.equal(other.lam, layer.lam) and other.lam.dtype == torch.float32
    assert copy.deepcopy(layer).half().lam.dtype == torch.float32
    empty = layer.to("meta")
    assert empty.lam.device.type == "meta" and empty.lam.dtype == torch.float32
    empty.to_empty(device="cpu")
    assert empty.lam.device.type == "cpu" and empty.lam.dtype == torch.float32
