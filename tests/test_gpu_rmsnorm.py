"""The root-mean-square norm on the GPU against its formula in fp64.

Tolerances.  A mean of squares in fp32 is off by at most 40 units of 2^-24 for a row of up to 32768
elements (8 to 32 additions in a thread, 10 across threads) and longer rows by 1 + C / 8192 more;
rstd by half of that and 3 units, y by 3 more: 2e-6 (34 units) of each value, 1e-5 for longer rows.
Gradients are of the same kind, relative to the largest sum of magnitudes; dw adds up to 60 rows
in fp32, and the rest in fp64.  16-bit outputs add half a unit in their last place."""
import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
EPS = 1e-5


def close(name, got, want, mass=None, rel=2e-6):
    got, dt = got.detach().double().cpu(), got.dtype
    assert got.shape == want.shape, name
    base = want.abs() if mass is None else (mass.max() if mass.numel() else 0)
    bound = rel * base + HALF_ULP[dt] * want.abs() + TINY[dt]
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    assert (err <= bound).all(), "%s: error %.3g" % (name, float(err.max()))


def place(t, shift=0):
    flat = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
    flat[shift:] = t.flatten().cuda()
    return flat[shift:].view(t.shape)


def make(B, T, C, dtype="f32", residual="same", seed=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    rdt = torch.float32 if residual == "f32" else dt
    rand = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    s = {"x": rand(B, T, C).to(dt), "dy": rand(B, T, C).to(dt), "res": rand(B, T, C).to(rdt),
         "dtotal": rand(B, T, C).to(rdt)}
    s = {k: place(t, shift) for k, t in s.items()}
    s["w"] = rand(C).cuda()
    if residual == "none":
        s["res"] = s["dtotal"] = None
    return s


def wide64(t):
    return None if t is None else t.detach().double().cpu()


def check(s, what="", rel=2e-6):
    import aware_conv_amd as A
    print("\ncase rmsnorm %s" % (what,), flush=True)
    y, total, rstd = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS, save_rstd=True)
    kept = s["x"] if total is None else total
    g = A.rmsnorm_bwd(kept, s["w"], rstd, s["dy"], dtotal=s["dtotal"])
    q, scale, qtotal = A.rmsnorm_fwd_e4m3(s["x"], s["w"], residual=s["res"], eps=EPS)
    plain = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS)
    torch.cuda.synchronize()
    assert plain[2] is None and torch.equal(plain[0], y)
    if s["res"] is not None:
        # one addition in fp32, rounded once more where the residual has 16 bits
        assert torch.equal(total, (s["x"].float() + s["res"].float()).to(s["res"].dtype))
        assert torch.equal(qtotal, total)
    else:
        assert total is None and qtotal is None
    want, mass = ref.rmsnorm(wide64(kept), wide64(s["w"]), EPS, wide64(s["dy"]), wide64(s["dtotal"]))
    close("y", y, want["y"], rel=rel)
    close("rstd", rstd, want["rstd"], rel=rel)
    close("dx", g["dx"], want["dx"], mass["dx"], rel=rel)
    close("dresidual", g["dresidual"], want["dx"], mass["dx"], rel=rel)
    close("dw", g["dw"], want["dw"], mass["dw"], rel=2 * rel)
    top = want["y"].abs().amax(-1)
    close("scale", scale, top / 448, rel=rel)
    # codes: to nearest of the value the kernel has, which is `rel` off: half a step, and that
    have = q.double().cpu() * scale.double().cpu()[..., None]
    step = torch.ldexp(torch.ones_like(have), (torch.frexp(want["y"].abs() / (top[..., None] / 448)).exponent - 1)
                       .clamp(min=-6) - 3) * (top[..., None] / 448)
    assert ((have - want["y"]).abs() <= 0.5 * step + 4 * rel * top[..., None]).all()
    assert q.dtype is torch.float8_e4m3fn
    return y, total, rstd, g, q, scale


WIDTHS = [1, 2, 7, 8, 9, 63, 64, 65, 511, 512, 513, 999, 1024, 1025, 2047, 2048, 2049, 4096, 4097, 8192, 8193, 16384,
          16385, 32768]


@pytest.mark.parametrize("dtype,residual", [("f32", "none"), ("f32", "same"), ("f16", "none"), ("f16", "same"),
                                            ("f16", "f32"), ("bf16", "none"), ("bf16", "same"), ("bf16", "f32")])
@pytest.mark.parametrize("C", WIDTHS)
def test_widths(dtype, residual, C):
    check(make(2, 3, C, dtype, residual, seed=C), what=(dtype, residual, C))


@pytest.mark.parametrize("dtype,residual", [("f32", "same"), ("f16", "none"), ("bf16", "f32")])
@pytest.mark.parametrize("C", [32769, 40001, 100000])
def test_rows_read_again(dtype, residual, C):
    check(make(1, 3, C, dtype, residual, seed=C), what=(dtype, residual, C), rel=1e-5)


@pytest.mark.parametrize("B,T", [(1, 1), (5, 1), (1, 5), (3, 700), (1, 2049)])
def test_rows(B, T):
    for C in (5, 300, 2500):
        check(make(B, T, C, "bf16", "f32", seed=T), what=(B, T, C))


@pytest.mark.parametrize("dtype,residual", [("f32", "same"), ("f16", "same"), ("bf16", "f32")])
@pytest.mark.parametrize("shift", [1, 3])
def test_views(dtype, residual, shift):
    """Odd addresses and rows that are parts of wider ones."""
    import aware_conv_amd as A
    C = 77
    s = make(2, 9, C, dtype, residual, seed=shift, shift=shift)
    want = check(s, what=("views", dtype, shift))
    wide = place(torch.full((2, 9, 3 * C), 7.0, dtype=DT[dtype]), shift)
    x, y, dx = wide.chunk(3, dim=2)
    x.copy_(s["x"])
    got = A.rmsnorm_fwd(x, s["w"], residual=s["res"], eps=EPS, y=y, save_rstd=True)
    assert got[0] is y and torch.equal(y, want[0]) and torch.equal(got[1], want[1])
    g = A.rmsnorm_bwd(got[1], s["w"], got[2], s["dy"], dtotal=s["dtotal"], grads={"dx": dx})
    assert torch.equal(dx, want[3]["dx"]) and torch.equal(x, s["x"])
    codes = torch.zeros(2, 9, C + 5, dtype=torch.float8_e4m3fn, device="cuda")[..., 3:3 + C]
    q, scale, _ = A.rmsnorm_fwd_e4m3(x, s["w"], residual=s["res"], eps=EPS, y=codes)
    assert q is codes and torch.equal(q.float(), want[4].float()) and torch.equal(scale, want[5])


@pytest.mark.parametrize("C", [300, 2500, 40001])
def test_residual_updated_in_place(C):
    import aware_conv_amd as A
    s = make(2, 5, C, "bf16", "f32", seed=3)
    want = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS)
    quant = A.rmsnorm_fwd_e4m3(s["x"], s["w"], residual=s["res"], eps=EPS)
    stream = s["res"].clone()
    y, total, _ = A.rmsnorm_fwd(s["x"], s["w"], residual=stream, eps=EPS, total=stream)
    assert total is stream and torch.equal(stream, want[1]) and torch.equal(y, want[0])
    stream = s["res"].clone()
    q, scale, _ = A.rmsnorm_fwd_e4m3(s["x"], s["w"], residual=stream, eps=EPS, total=stream)
    assert torch.equal(stream, want[1]) and torch.equal(q.float(), quant[0].float()) and torch.equal(scale, quant[1])


def test_two_axes():
    import aware_conv_amd as A
    s = make(6, 1, 200, "bf16", "same", seed=3)
    want = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], save_rstd=True)
    got = A.rmsnorm_fwd(s["x"][:, 0], s["w"], residual=s["res"][:, 0], save_rstd=True)
    for a, b in zip(got, want):
        assert torch.equal(a, b[:, 0])
    g = A.rmsnorm_bwd(got[1], s["w"], got[2], s["dy"][:, 0])
    assert torch.equal(g["dx"], A.rmsnorm_bwd(want[1], s["w"], want[2], s["dy"])["dx"][:, 0])


def test_zeros_infinities_and_nan():
    """A row of zeros gives zeros (scale 0); one with a NaN or an infinity touches no other row."""
    import aware_conv_amd as A
    s = make(1, 4, 300, "f32", "none", seed=1)
    s["x"][0, 0] = 0
    s["x"][0, 1, 7] = float("nan")
    s["x"][0, 2, 9] = float("inf")
    y, _, rstd = A.rmsnorm_fwd(s["x"], s["w"], eps=EPS, save_rstd=True)
    q, scale, _ = A.rmsnorm_fwd_e4m3(s["x"], s["w"], eps=EPS)
    assert (y[0, 0] == 0).all() and (q[0, 0].float() == 0).all() and scale[0, 0] == 0
    assert y[0, 1].isnan().all() and q[0, 1].float().isnan().all()
    assert y[0, 2, 9].isnan() and q[0, 2, 9].float().isnan() and (y[0, 2, :9] == 0).all()
    assert y[0, 3].isfinite().all() and q[0, 3].float().isfinite().all()
    assert torch.equal(y[0, 3:], A.rmsnorm_fwd(s["x"][:, 3:].contiguous(), s["w"], eps=EPS)[0][0])


@pytest.mark.parametrize("scale", [1e-18, 1e-4, 1e4, 1e15])
def test_sizes_of_values(scale):
    """Squares from 1e-36, far below eps, to 1e30."""
    s = make(1, 3, 300, "f32", "none", seed=1)
    s["x"] *= scale
    check(s, what=("size", scale))


def test_more_rows_than_a_launch_has_threads_for():
    import aware_conv_amd as A
    n = (1 << 26) + 5
    x = torch.ones(n, 1, dtype=torch.float16, device="cuda")
    x[-3:, 0] = torch.tensor([2.0, 0.0, -3.0])
    w = torch.full((1,), 0.5, device="cuda")
    y, _, rstd = A.rmsnorm_fwd(x, w, eps=0.0, save_rstd=True)
    assert (y[:-3] == 0.5).all() and (rstd[:-3] == 1).all()
    assert y[-3:, 0].nan_to_num(9).tolist() == [0.5, 9.0, -0.5]  # a row of zeros without eps has no norm
    dw = A.rmsnorm_bwd(x[:-3], w, rstd[:-3], y[:-3])["dw"]
    # halves are added exactly, and their sum, 33554433, is rounded: fp32 has every fourth number there
    assert dw.item() == torch.tensor((n - 3) * 0.5, dtype=torch.float32).item()


@pytest.mark.parametrize("top", [1e-30, 1e-36, 2e-38, 1e-42, 0.0])
def test_scales_of_small_rows(top):
    """Down to where the scale leaves the normal numbers, and the row is zero."""
    import aware_conv_amd as A
    x = torch.ones(1, 1, 100, device="cuda")
    x[0, 0, ::3] = 0
    w = torch.full((100,), top, device="cuda")
    q, scale, _ = A.rmsnorm_fwd_e4m3(x, w, eps=0.0)
    y = A.rmsnorm_fwd(x, w, eps=0.0)[0]
    assert torch.isfinite(q.float()).all()
    if float(y.max()) / 448 >= 2.0 ** -126:
        # the largest is coded as 448: what the scale rounds to is all that is off
        assert ((q.double() * scale.double()[..., None] - y.double()).abs() <= 2.0 ** -22 * y.double()).all()
    else:
        assert scale.item() == 0 and (q.float() == 0).all()


def test_into_a_product_in_8_bits():
    """As it is used: codes and scales of rows into a product whose weights are coded by rows too.
    Both are off by at most 2^-4 of each value, mean 2^-5.5 of either sign: 0.04 of the result's
    size covers the sum of 256 such terms."""
    import aware_conv_amd as A
    s = make(1, 40, 256, "bf16", "f32", seed=1)
    weight = torch.randn(512, 256, device="cuda")
    size = weight.abs().amax(1, keepdim=True) / 448
    codes = (weight / size).to(torch.float8_e4m3fn)
    q, scale, total = A.rmsnorm_fwd_e4m3(s["x"], s["w"], residual=s["res"])
    got = torch._scaled_mm(q[0], codes.t(), scale_a=scale[0][:, None], scale_b=size.t(), out_dtype=torch.bfloat16)
    want = A.rmsnorm_fwd(s["x"].float(), s["w"], residual=s["res"])[0][0] @ weight.t()
    assert (got.float() - want).norm() <= 0.04 * want.norm()


def test_no_rows():
    import aware_conv_amd as A
    for B, T, C in ((0, 3, 20), (2, 0, 20), (2, 3, 0)):
        s = make(B, T, C, "bf16", "f32")
        y, total, rstd = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], save_rstd=True)
        g = A.rmsnorm_bwd(total, s["w"], rstd, s["dy"])
        assert y.shape == (B, T, C) and (g["dw"] == 0).all() and g["dw"].shape == (C,)


def test_offsets_beyond_32_bits():
    import aware_conv_amd as A
    s = make(2, 5, 300, "bf16", "same", seed=2)
    want = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"])
    far = torch.zeros((1 << 31) + 5000, dtype=torch.bfloat16, device="cuda").as_strided((2, 5, 300), (1 << 31, 400, 1))
    far.copy_(s["x"])
    got = A.rmsnorm_fwd(far, s["w"], residual=s["res"])
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_captured_calls():
    import aware_conv_amd as A
    s = make(2, 700, 300, "bf16", "f32", seed=1)

    def run():
        y, total, rstd = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], save_rstd=True)
        q, scale, _ = A.rmsnorm_fwd_e4m3(s["x"], s["w"], residual=s["res"])
        g = A.rmsnorm_bwd(total, s["w"], rstd, s["dy"], dtotal=s["dtotal"])
        return [y, total, q.view(torch.uint8), scale, g["dx"], g["dresidual"], g["dw"]]

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for _ in range(4):
        for n in ("x", "dy", "res", "dtotal"):
            s[n].copy_(torch.randn(s[n].shape, device="cuda"))
        want = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip(kept, want):
            assert torch.equal(a, b)


@pytest.mark.parametrize("dtype,residual", [("f32", "none"), ("f32", "same"), ("bf16", "same"), ("bf16", "f32")])
@pytest.mark.parametrize("use", ["both", "y", "total"])
def test_autograd(dtype, residual, use):
    import aware_conv_amd as A
    if residual == "none" and use != "y":
        return
    s = make(2, 50, 120, dtype, residual, seed=7)
    p = {"x": s["x"], "w": s["w"], "residual": s["res"]}
    p = {k: t.detach().clone().requires_grad_() for k, t in p.items() if t is not None}
    y, total = A.rms_norm(eps=EPS, **p)
    loss = 0
    if use != "total":
        loss = loss + (y * s["dy"]).float().sum()
    if use != "y":
        loss = loss + (total * s["dtotal"]).float().sum()
    loss.backward()
    dy = wide64(s["dy"]) if use != "total" else torch.zeros(2, 50, 120, dtype=torch.float64)
    want, mass = ref.rmsnorm(wide64(p["x"] if total is None else total), wide64(s["w"]), EPS, dy,
                             wide64(s["dtotal"]) if use != "y" else None)
    close("x", p["x"].grad, want["dx"], mass["dx"])
    close("w", p["w"].grad, want["dw"], mass["dw"], rel=4e-6)
    if "residual" in p:
        close("residual", p["residual"].grad, want["dx"], mass["dx"])


def test_gradients_against_differences():
    """Along a random direction, of a loss summed in fp64: see the scan's test of the same name."""
    import aware_conv_amd as A
    s = make(2, 20, 50, "f32", "same", seed=11)
    p = {k: t.detach().clone().requires_grad_() for k, t in (("x", s["x"]), ("w", s["w"]), ("residual", s["res"]))}
    y, total = A.rms_norm(**p)
    ((y * s["dy"]).sum() + (total * s["dtotal"]).sum()).backward()

    def loss(q):
        y, total = A.rms_norm(**q)
        return float((y.double() * s["dy"].double()).sum() + (total.double() * s["dtotal"].double()).sum())

    y = y.detach()
    size = float((y.double() * s["dy"].double()).abs().sum() + (total.detach().double() * s["dtotal"].double()).abs().sum())
    for k in p:
        torch.manual_seed(1)
        way = torch.randn_like(p[k])
        at = {n: t.detach() for n, t in p.items()}
        up, down = (loss({**at, k: at[k] + sign * 2 ** -7 * way}) for sign in (1, -1))
        slope = float((p[k].grad.double() * way.double()).sum())
        assert abs((up - down) * 2 ** 6 - slope) <= 1e-3 * size, k
