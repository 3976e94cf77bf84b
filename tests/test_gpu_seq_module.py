"""GatedScan2d converted to another dtype, on the GPU."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("convert", [lambda m: m.half(), lambda m: m.to("cuda", torch.float16)])
def test_a_converted_layer_runs_as_one_made_so(convert):
    import aware_conv_amd as A
    torch.manual_seed(0)
    layer = A.GatedScan2d(6, kernel_size=3, levels=1, device="cuda")
    made = A.GatedScan2d(6, kernel_size=3, levels=1, device="cuda", dtype=torch.float16)
    made.load_state_dict(layer.state_dict())
    layer = convert(layer)
    x = torch.randn(2, 6, 8, 8, device="cuda", dtype=torch.float16)
    out = []
    for m in (layer, made):
        y = m(x)
        y.float().square().mean().backward()
        out.append([y.detach()] + [p.grad for p in m.parameters()])
    assert all(torch.equal(a, b) for a, b in zip(*out)) and layer.lam.grad.dtype == torch.float32
