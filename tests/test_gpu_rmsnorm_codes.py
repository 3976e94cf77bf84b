"""The norm's 8-bit codes to the bit.  Rows of ones have a root mean square of exactly 1, so that
y is the weight itself, and the weights here lie on and next to the ties between two codes."""
import pytest
import torch

pytestmark = pytest.mark.gpu

CODES = torch.arange(0x7f, dtype=torch.uint8).view(torch.float8_e4m3fn).float()  # 0 to 448


def by_formula(y, scale):
    """The fp32 product with the inverse in e4m3, to nearest even, by the processor."""
    return (y * (1 / scale)).clamp(-448, 448).to(torch.float8_e4m3fn)


def near_ties(top, count, g):
    """`count` values of at most `top`, up to two places from where y / (top / 448) is between two codes."""
    scale = torch.tensor(top) / 448
    tie = (CODES[1:] + CODES[:-1]) / 2
    y = (tie[torch.randint(len(tie), (count,), generator=g)] * scale).clone()
    y = (y.view(torch.int32) + torch.randint(-2, 3, (count,), generator=g, dtype=torch.int32)).view(torch.float32)
    y *= 1 - 2 * torch.randint(2, (count,), generator=g)
    y[0] = top
    return y.clamp(-top, top), scale


@pytest.mark.parametrize("top", [1.7, 300.0, 3.3e-5, 7.7e30, 6e-36])
@pytest.mark.parametrize("C,dtype", [(500, torch.float32), (2048, torch.bfloat16), (4097, torch.float16),
                                     (20000, torch.bfloat16), (40001, torch.float32)])
def test_codes_next_to_ties(C, dtype, top):
    """To the bit; and no further from the quotient than half a step and two roundings of 2^-24, with
    that of the quotient itself 2^-22 in all."""
    import aware_conv_amd as A
    print("\ncase codes %s" % ((C, dtype, top),), flush=True)
    g = torch.Generator().manual_seed(C)
    x = torch.ones(1, 1, C, dtype=dtype, device="cuda")
    for _ in range(8):
        w, scale = near_ties(top, C, g)
        q, got, _ = A.rmsnorm_fwd_e4m3(x, w.cuda(), eps=0.0)
        q = q[0, 0].cpu()
        assert got.item() == scale.item()
        assert torch.equal(q.view(torch.uint8), by_formula(w, scale).view(torch.uint8))
        want = w.double() / scale.double()
        step = torch.ldexp(torch.ones_like(want), (torch.frexp(want.abs()).exponent - 1).clamp(min=-6) - 3)
        assert ((q.double() - want).abs() <= step / 2 + 2.0 ** -22 * want.abs()).all()


def test_codes_of_random_rows():
    """y from the sum, rstd and w in the header's order, in fp32."""
    import aware_conv_amd as A
    g = torch.Generator().manual_seed(0)
    x = torch.randn(1, 2048, 2048, generator=g).bfloat16()
    res = torch.randn(1, 2048, 2048, generator=g)
    w = torch.randn(2048, generator=g)
    at = {"residual": res.cuda(), "eps": 1e-5}
    _, total, rstd = A.rmsnorm_fwd(x.cuda(), w.cuda(), save_rstd=True, **at)
    q, scale, _ = A.rmsnorm_fwd_e4m3(x.cuda(), w.cuda(), **at)
    y = total.cpu() * rstd.cpu()[..., None] * w
    assert torch.equal(scale.cpu(), y.abs().amax(-1) / 448)
    assert torch.equal(q.cpu().view(torch.uint8), by_formula(y, scale.cpu()[..., None]).view(torch.uint8))
