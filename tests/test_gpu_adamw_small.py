"""The AdamW step where something in it is small."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype,bits", [(torch.float32, 32), (torch.float32, 8), (torch.bfloat16, 32)])
@pytest.mark.parametrize("lr", [1e-5, 1e-6])
def test_slow_weight_decay(lr, dtype, bits):
    """lr * weight_decay of 1e-7 and 1e-8, at and below the spacing of fp32 under 1: with and
    without it, a million parameters differ on the mean by what 50 steps take off.  Each step
    rounds a parameter of 0.1 to 0.2 by at most 7.5e-9, evenly, as its update is spread over many
    units: 4e-9 * sqrt(2 * 50) / 1024 = 4e-11 of noise on the mean, 6e-5 and 6e-4 of the 7.5e-7
    and 7.5e-8 that are taken off; ten times that is allowed."""
    import aware_conv_amd as A
    print("\ncase decay %s" % ((lr, dtype, bits),), flush=True)
    n, steps, decay = 1 << 20, 50, 0.01
    ends, path = [], []
    for wd in (decay, 0.0):
        g = torch.Generator(device="cuda").manual_seed(1)
        w = 0.1 + 0.1 * torch.rand(n, generator=g, device="cuda")
        masters = None if dtype == torch.float32 else [w]
        p = w if masters is None else w.to(dtype)
        if bits == 8:
            codes = torch.randint(48, 120, (2, n), generator=g, device="cuda", dtype=torch.uint8)
            m, v = (c.view(torch.float8_e4m3fn) for c in codes)
            scales = [torch.full((n // 256,), 1e-5, device="cuda")], [torch.full((n // 256,), 1e-5, device="cuda")]
        else:
            m = torch.randn(n, generator=g, device="cuda") * 1e-3
            v = 1e-6 * (0.5 + torch.rand(n, generator=g, device="cuda"))
            scales = None
        step = torch.full((1,), 100, dtype=torch.int32, device="cuda")
        for _ in range(steps):
            path.append(float(w.double().mean()))  # which the updates move, too
            grad = (torch.randn(n, generator=g, device="cuda") * 1e-3).to(dtype)
            A.adamw_step([p], [grad], [m], [v], step, lr=lr, weight_decay=wd, masters=masters, scales=scales)
        ends.append(w.double())
    # the moments do not depend on the parameters: the updates are the same
    want = -lr * decay * sum(path[:steps])
    got = float((ends[0] - ends[1]).mean())
    assert abs(got / want - 1) <= 6e-9 / lr


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("size", [1e-16, 1e-17, 1e-18, 1e-19, 1e-20])
def test_gradients_whose_squares_leave_the_normal_range(size, bits):
    """Without eps the first step moves a parameter by lr, whatever the gradient: v is exact to
    1e-6 of itself and 2^-149 (its spacing below 2^-126, two roundings), and its root to half."""
    import aware_conv_amd as A
    print("\ncase tiny %s" % ((size, bits),), flush=True)
    n = 300
    p = torch.zeros(n, device="cuda")
    g = torch.full((n,), size, device="cuda")
    if bits == 8:
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        scales = [torch.zeros(2, device="cuda")], [torch.zeros(2, device="cuda")]
    else:
        m, v, scales = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda"), None
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    A.adamw_step([p], [g], [m], [v], step, lr=1e-3, eps=0.0, weight_decay=0.0, scales=scales)
    bound = 1e-3 * (2e-6 + 2.0 ** -150 / (1e-3 * size ** 2))
    assert ((p.double() + 1e-3).abs() <= bound).all()


def test_moments_near_the_largest_float():
    """3.3e38 is finite: it is the largest of its block, and sets its scale.  Codes are exact: the
    scale is 3.3e38 / 448 to fp32, and every other magnitude of the block is 0 of it."""
    import aware_conv_amd as A
    g = torch.ones(256, device="cuda")
    g[7], g[9] = -3.3e38, float("inf")
    m, v = (torch.zeros(256, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
    scales = [torch.zeros(1, device="cuda")], [torch.zeros(1, device="cuda")]
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    A.adamw_step([torch.zeros(256, device="cuda")], [g], [m], [v], step, betas=(0.0, 0.999), scales=scales)
    assert abs(float(scales[0][0]) / (3.3e38 / 448) - 1) <= 2.0 ** -23
    got = m.float().cpu()
    assert got[7] == -448 and got[9].isnan()
    got[7] = got[9] = 0
    # 1 of a scale of 7e35 is 0 or, for a dither that rounds it up, the lowest code
    assert ((got == 0) | (got == 2.0 ** -9)).all()
