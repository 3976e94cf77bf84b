"""The block of norm, convolution and scan under autocast: trained, and served from a cache that was
made with or without it."""
import pytest
import torch

pytestmark = pytest.mark.gpu

BF16 = {"device_type": "cuda", "dtype": torch.bfloat16}


def blocks(dtype=torch.float32):
    import aware_conv_amd as A
    torch.manual_seed(0)
    made = [A.SelectiveMixer(24, states=5, rank=3, device="cuda", dtype=dtype, residual_fp32=True) for _ in range(2)]
    with torch.no_grad():
        for m in made:
            m.conv_b.normal_()
    return made


def through(made, x, call):
    y, res = x, None
    for k, m in enumerate(made):
        y, res = call(k, m, y, res)
    return y.float() + res


@pytest.mark.parametrize("inside", [True, False])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_served_under_autocast(dtype, inside):
    """A padded prompt, then single positions, against one pass over each whole sequence: 16-bit
    intermediate results, rounded by 2^-8 in other groupings."""
    print("\ncase autocast %s %s" % (dtype, inside), flush=True)
    made = blocks(dtype)
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 40, 24, generator=g).to(dtype).cuda()
    with torch.autocast(enabled=inside, **BF16):
        caches = [m.new_cache(5) for m in made]
    rows, lengths = [4, 0, 2], [20, 3, 9]
    n = torch.tensor(lengths, dtype=torch.int32, device="cuda")
    slots = torch.tensor(rows, dtype=torch.int32, device="cuda")
    with torch.no_grad(), torch.autocast(**BF16):
        want = through(made, x, lambda k, m, y, r: m(y, r))
        top = want.abs().max()
        got = through(made, x[:, :20], lambda k, m, y, r: m.prompt(y, caches[k], r, lengths=n, rows=rows))
        for i, k in enumerate(lengths):
            assert (got[i, :k] - want[i, :k]).abs().max() <= 0.05 * top
        for step in range(20):
            at = torch.stack([x[i, k + step] for i, k in enumerate(lengths)])
            got = through(made, at, lambda k, m, y, r: m.step(y, caches[k], r, slots=slots))
            for i, k in enumerate(lengths):
                assert (got[i] - want[i, k + step]).abs().max() <= 0.05 * top, (step, i)


def test_a_cache_in_the_layers_type_holds_what_autocast_gives():
    """The inputs that an fp32 cache holds are 16-bit values, so steps from it and from a cache of
    that type are the same: the convolution rounds once either way."""
    m = blocks()[0]
    g = torch.Generator(device="cuda").manual_seed(2)
    wide = m.new_cache(3)
    narrow = (wide[0].bfloat16(), wide[1].clone())
    with torch.autocast(**BF16):
        for _ in range(6):
            x = torch.randn(3, 24, generator=g, device="cuda")
            a, b = m.step(x, wide), m.step(x, narrow)
            assert a[0].dtype is torch.bfloat16 and torch.equal(a[0], b[0])
    assert torch.equal(wide[0], narrow[0].float()) and torch.equal(wide[1], narrow[1])


def test_gradients_under_autocast():
    m = blocks()[0]
    x = torch.randn(2, 30, 24, device="cuda", requires_grad=True)
    with torch.autocast(**BF16):
        out, total = m(x)
    (out.float() + total).square().mean().backward()
    for name, p in [*m.named_parameters(), ("x", x)]:
        assert p.grad.dtype is torch.float32 and p.grad.isfinite().all(), name
