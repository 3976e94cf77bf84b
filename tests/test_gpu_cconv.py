"""The causal convolution on the GPU against its formula in fp64.

Tolerances.  A sum of K products in fp32 is off by at most (K + 1) 2^-24 of the sum of its terms'
magnitudes, and the gate and its slope by a few units more; sums over positions are of terms of
either sign, added in fp32 over runs of up to 256 positions and in fp64 beyond: 2e-6 of the
largest sum of magnitudes covers both (32 units of 2^-24).  16-bit outputs add half a unit in
their last place."""
import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def close(name, got, want, mass):
    got, dt = got.detach().double().cpu(), got.dtype
    assert got.shape == want.shape, name
    top = float(mass.max()) if mass.numel() else 0.0
    bound = 2e-6 * top + HALF_ULP[dt] * want.abs() + TINY[dt]
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    assert (err <= bound).all(), "%s: error %.3g, largest sum of magnitudes %.3g" % (name, float(err.max()), top)


def place(t, shift=0):
    flat = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
    flat[shift:] = t.flatten().cuda()
    return flat[shift:].view(t.shape)


def make(B, T, C, K, dtype="f32", seed=0, without=(), packed=False, shift=0):
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    rand = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    s = {"x": rand(B, T, C).to(dt), "dy": rand(B, T, C).to(dt), "h0": rand(B, K - 1, C).to(dt),
         "dlast": rand(B, K - 1, C).to(dt)}
    if packed:
        s["x"] = place(torch.cat([s["x"], rand(B, T, C).to(dt)], 2), shift).chunk(2, dim=2)[0]
    s = {k: t if t.is_cuda else place(t, shift) for k, t in s.items()}
    s["w"], s["bias"] = rand(C, K).cuda(), rand(C).cuda()
    for k in without:
        s[k] = None
    return s


def wide64(t):
    return None if t is None else t.detach().double().cpu()


def check(s, lengths=None, silu=True, what=""):
    import aware_conv_amd as A
    print("\ncase cconv %s" % (what,), flush=True)
    form = {"bias": s["bias"], "h0": s["h0"], "silu": silu,
            "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    y, last = A.cconv_fwd(s["x"], s["w"], **form)
    g = A.cconv_bwd(s["x"], s["w"], s["dy"], dlast=s["dlast"], **form)
    torch.cuda.synchronize()
    r = {k: wide64(s[k]) for k in s}
    if lengths is not None:
        for i, n in enumerate(ref.counts(*s["x"].shape[:2], lengths)):
            r["x"][i, n:], r["dy"][i, n:] = 0, 0
    want, mass = ref.cconv(lengths=lengths, act=silu, **r)
    close("y", y, want["y"], mass["y"])
    assert torch.equal(last.double().cpu(), want["last"])
    for k in ("dx", "dw", "dbias", "dh0"):
        if k == "dbias" and s["bias"] is None:
            assert g[k] is None
        else:
            close(k, g[k], want[k], mass[k])
    return y, last, g


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 7, 8, 9, 15, 16, 17, 31, 32, 33, 64, 127, 129, 256, 257, 600])
def test_lengths(dtype, T):
    check(make(2, T, 5, 4, dtype=dtype, seed=T), what=(dtype, T))


@pytest.mark.parametrize("K", [1, 2, 3, 4, 5, 6, 7, 8])
@pytest.mark.parametrize("silu", [True, False])
def test_taps(K, silu):
    for T in (1, 3, 6, 40, 300):
        check(make(2, T, 9, K, dtype="f32", seed=K), silu=silu, what=("taps", K, T, silu))
    check(make(2, 40, 9, K, dtype="bf16", seed=K), silu=silu, what=("taps", K, "bf16", silu))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("C", [1, 2, 3, 4, 7, 8, 9, 31, 127, 128, 129, 255, 256, 257, 999])
def test_channels(dtype, C):
    check(make(2, 21, C, 4, dtype=dtype, seed=C), what=(dtype, C))


@pytest.mark.parametrize("without", [("bias",), ("h0",), ("dlast",), ("bias", "h0", "dlast")])
def test_absent_terms(without):
    check(make(2, 50, 20, 4, seed=3, without=without), what=without)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("K", [2, 4, 8])
@pytest.mark.parametrize("T", [9, 40, 600])
def test_ragged(dtype, K, T):
    """Lengths of zero, one, fewer than the taps, the ends of runs, beyond T and below 0; NaN where
    nothing is read."""
    lengths = [T, 0, 1, 2, 3, 7, 8, 16, 31, 32, 33, 255, 256, -5, T + 9, T - 1]
    s = make(len(lengths), T, 7, K, dtype=dtype, seed=T)
    for i, n in enumerate(ref.counts(len(lengths), T, lengths)):
        s["x"][i, n:], s["dy"][i, n:] = float("nan"), float("nan")
    y, _, g = check(s, lengths, what=("ragged", dtype, K, T))
    for i, n in enumerate(ref.counts(len(lengths), T, lengths)):
        assert (y[i, n:] == 0).all() and (g["dx"][i, n:] == 0).all()
    s["h0"] = None
    check(s, lengths, what=("ragged, no inputs before", dtype, K, T))


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_views(dtype, shift):
    import aware_conv_amd as A
    s = make(2, 45, 19, 4, dtype=dtype, seed=shift, packed=True, shift=shift)
    y, _, g = check(s, what=("views", dtype, shift))
    wide = place(torch.full((2, 45, 3 * 19), 7.0, dtype=DT[dtype]), shift)
    dx = wide[..., 19:38]
    again = A.cconv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], h0=s["h0"], dlast=s["dlast"], grads={"dx": dx})
    for k in g:
        assert torch.equal(again[k], g[k]), k
    assert (wide[..., :19] == 7).all() and (wide[..., 38:] == 7).all() and again["dx"] is dx


def test_no_positions():
    import aware_conv_amd as A
    s = make(2, 0, 5, 4, seed=1)
    y, last = A.cconv_fwd(s["x"], s["w"], h0=s["h0"])
    assert y.shape == (2, 0, 5) and torch.equal(last, s["h0"])
    g = A.cconv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], h0=s["h0"], dlast=s["dlast"])
    assert torch.equal(g["dh0"], s["dlast"]) and (g["dw"] == 0).all() and (g["dbias"] == 0).all()


def test_offsets_beyond_32_bits():
    import aware_conv_amd as A
    s = make(2, 50, 33, 4, dtype="bf16", seed=2)
    want = A.cconv_fwd(s["x"], s["w"], bias=s["bias"])
    far = torch.zeros((1 << 31) + 50 * 40, dtype=torch.bfloat16, device="cuda").as_strided((2, 50, 33), (1 << 31, 40, 1))
    far.copy_(s["x"])
    y = torch.zeros(50 * (1 << 26), dtype=torch.bfloat16, device="cuda").as_strided((2, 50, 33), (64, 1 << 26, 1))
    got = A.cconv_fwd(far, s["w"], bias=s["bias"], y=y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_two_runs_agree_bit_for_bit():
    s = make(3, 900, 70, 4, dtype="bf16", seed=8)
    a, b = check(s, what="first"), check(s, what="second")
    for k in a[2]:
        assert torch.equal(a[2][k], b[2][k]), k


def test_large_values():
    """Where silu saturates on either side, its slope too."""
    s = make(1, 60, 8, 4, seed=5)
    s["x"] *= torch.logspace(-3, 4, 60, device="cuda")[None, :, None]
    check(s, what="large")


def test_captured_calls():
    import aware_conv_amd as A
    s = make(2, 300, 70, 4, dtype="bf16", seed=1)

    def run():
        return A.cconv_fwd(s["x"], s["w"], bias=s["bias"], h0=s["h0"]), A.cconv_bwd(
            s["x"], s["w"], s["dy"], bias=s["bias"], h0=s["h0"], dlast=s["dlast"])

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for _ in range(4):
        for n in ("x", "dy", "h0"):
            s[n].copy_(torch.randn(s[n].shape, device="cuda"))
        (y, last), g = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept[0][0], y) and torch.equal(kept[0][1], last)
        for n in g:
            assert torch.equal(kept[1][n], g[n]), n


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,C,K", [(1, 1, 1), (1, 5, 2), (3, 17, 4), (5, 130, 3), (70, 33, 8), (1, 384, 4)])
@pytest.mark.parametrize("silu", [True, False])
def test_step(dtype, B, C, K, silu):
    import aware_conv_amd as A
    print("\ncase cconv step %s" % ((dtype, B, C, K, silu),), flush=True)
    s = make(B, 1, C, K, dtype=dtype, seed=C, packed=True)
    S = B + 3
    cache = torch.randn(S, K - 1, C, device="cuda").to(DT[dtype])
    before = cache.clone()
    slots = torch.randperm(S)[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, S  # passed over
    on = [i for i in range(B) if 0 <= slots[i] < S]
    at = [int(slots[i]) for i in on]
    y = A.cconv_step(s["x"][:, 0], s["w"], cache, bias=s["bias"], slots=slots.cuda(), silu=silu)
    h0 = before.double().cpu()[slots.long().clamp(0, S - 1)]
    want, mass = ref.cconv(wide64(s["x"]), wide64(s["w"]), wide64(s["bias"]), h0=h0, act=silu)
    close("y", y[on], want["y"][on, 0], mass["y"][on, 0])
    assert torch.equal(cache[at].double().cpu(), want["last"][on])
    rest = [k for k in range(S) if k not in at]
    assert torch.equal(cache[rest], before[rest])
    assert (y[[i for i in range(B) if i not in on]] == 0).all()


def test_positions_one_by_one():
    """A prompt at once and single positions after it give what one pass gives, to the bit: the
    same sums in the same order."""
    import aware_conv_amd as A
    s = make(3, 30, 40, 4, dtype="bf16", seed=1)
    whole, last = A.cconv_fwd(s["x"], s["w"], bias=s["bias"])
    y, cache = A.cconv_fwd(s["x"][:, :2], s["w"], bias=s["bias"])
    parts = [y] + [A.cconv_step(s["x"][:, t], s["w"], cache, bias=s["bias"])[:, None] for t in range(2, 30)]
    assert torch.equal(torch.cat(parts, 1), whole) and torch.equal(cache, last)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("use", ["both", "y", "last"])
def test_autograd(dtype, use):
    import aware_conv_amd as A
    s = make(2, 50, 20, 4, dtype=dtype, seed=7)
    p = {k: s[k].detach().clone().requires_grad_() for k in ("x", "w", "bias", "h0")}
    y, last = A.causal_conv(**p)
    loss = 0
    if use != "last":
        loss = loss + (y * s["dy"]).float().sum()
    if use != "y":
        loss = loss + (last * s["dlast"]).float().sum()
    loss.backward()
    r = {k: wide64(s[k]) for k in s}
    if use == "last":
        r["dy"] = torch.zeros_like(r["dy"])
    if use == "y":
        r["dlast"] = None
    want, mass = ref.cconv(**r)
    for k, n in (("x", "dx"), ("w", "dw"), ("bias", "dbias"), ("h0", "dh0")):
        close(k, p[k].grad, want[n], mass[n])


def test_gradients_against_differences():
    """Along a random direction, of a loss summed in fp64: see the scan's test of the same name."""
    import aware_conv_amd as A
    s = make(2, 40, 18, 4, seed=11)
    p = {k: s[k].detach().clone().requires_grad_() for k in ("x", "w", "bias", "h0")}
    y, last = A.causal_conv(**p)
    (y * s["dy"]).sum().backward()

    def loss(q):
        return float((A.causal_conv(**q)[0].double() * s["dy"].double()).sum())

    y = y.detach()
    size = float((y.double() * s["dy"].double()).abs().sum())
    for k in p:
        torch.manual_seed(1)
        way = torch.randn_like(p[k])
        at = {n: t.detach() for n, t in p.items()}
        up, down = (loss({**at, k: at[k] + sign * 2 ** -7 * way}) for sign in (1, -1))
        slope = float((p[k].grad.double() * way.double()).sum())
        assert abs((up - down) * 2 ** 6 - slope) <= 1e-3 * size, k
