"""The gated linear recurrence on the GPU against its formulas in fp64.

Tolerances.  An element's gates are formed to a few units of 2^-24; a state
adds such an error at each step and forgets it with the decay, at most 0.999
here: about 1000 steps, errors of either sign, so about sqrt(500) * 2 * 6e-8 =
3e-6 of the states' size, and 1e-5 of the tensor's largest value at four
times that (the bound that the layer's fp32 tests use).  16-bit outputs add
half a unit in their last place.  dlam adds up many terms of both signs: 1e-5
of the sum of their magnitudes."""
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}


def close(name, got, want, mass=None):
    got, dt = got.detach().double().cpu(), got.dtype
    assert got.shape == want.shape, name
    top = float(want.abs().max()) if want.numel() else 0.0
    bound = 1e-5 * (mass if mass is not None else top) + HALF_ULP[dt] * want.abs() + TINY[dt]
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    assert (err <= bound).all(), "%s: error %.3g, largest value %.3g" % (name, float(err.max()), top)


def make(B, C, T, dtype, layout, seed, packed=False, shift=0):
    """x, r, i, dh as the kernels take them (views of a projection, or `shift` elements off their
    allocation) and lam, h0, dh_last."""
    g = torch.Generator().manual_seed(seed)
    shape = (B, C, T) if layout == "bct" else (B, T, C)
    dt = DT[dtype]

    def place(t):
        flat = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
        flat[shift:] = t.flatten().cuda()
        return flat[shift:].view(t.shape)

    if packed:
        dim = 1 if layout == "bct" else 2
        wide = list(shape)
        wide[dim] = 3 * C
        x, r, i = place(torch.randn(wide, generator=g).to(dt)).chunk(3, dim=dim)
    else:
        x, r, i = (place(torch.randn(shape, generator=g).to(dt)) for _ in range(3))
    dh = place(torch.randn(shape, generator=g).to(dt))
    a = 0.5 + 0.499 * torch.rand(C, generator=g, dtype=torch.float64)
    lam = torch.log(torch.expm1(-torch.log(a) / 8)).float()
    return {"x": x, "r": r, "i": i, "dh": dh, "lam": lam.cuda(),
            "h0": torch.randn(B, C, generator=g).cuda(),
            "dh_last": torch.randn(B, C, generator=g).cuda()}


def bct(t, layout):
    t = t.detach().double().cpu()
    t = t.flatten(2) if t.dim() == 4 else t
    return t if layout == "bct" else t.transpose(1, 2)


def check(d, layout, lengths=None, reverse=False, state=True, grads=None, what=""):
    import aware_conv_amd as A
    print("\ncase gscan %s" % (what,), flush=True)
    form = {"layout": layout, "reverse": reverse,
            "lengths": None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")}
    h0, dh_last = (d["h0"], d["dh_last"]) if state else (None, None)
    h, h_last, states = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"], h0=h0, save_states=True, **form)
    plain = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"], h0=h0, **form)
    out = A.gscan_bwd(d["x"], d["r"], d["i"], d["lam"], states, d["dh"], dh_last=dh_last,
                      grads=grads, **form)
    torch.cuda.synchronize()
    assert plain[2] is None
    assert torch.equal(plain[0], h) and torch.equal(plain[1], h_last)
    args = [bct(d[k], layout) for k in ("x", "r", "i")] + [d["lam"].double().cpu()]
    rh0 = None if not state else d["h0"].double().cpu()
    rdl = None if not state else d["dh_last"].double().cpu()
    rf = {"lengths": lengths, "reverse": reverse}
    if lengths is not None:  # what lies beyond the lengths is not read
        for b, n in enumerate(lengths):
            for t in args[:3]:
                t[b, :, max(n, 0):] = 0
    wh, wl, _ = ref.fwd(*args, h0=rh0, **rf)
    wg = ref.bwd(*args, torch.nan_to_num(bct(d["dh"], layout)), h0=rh0, dh_last=rdl, **rf)
    close("h", bct(h, layout).to(h.dtype), wh)
    close("h_last", h_last, wl)
    for n in ("dx", "dr", "di"):
        close(n, bct(out[n], layout).to(h.dtype), wg[n])
    close("dh0", out["dh0"], wg["dh0"])
    close("dlam", out["dlam"], wg["dlam"], mass=wg["mass"])
    return h, out


LENGTHS = [1, 2, 4, 5, 63, 64, 65, 196, 256, 257, 511, 513, 1300]


@pytest.mark.parametrize("layout", ["bct", "btc"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", LENGTHS)
def test_lengths(layout, dtype, T):
    check(make(2, 3, T, dtype, layout, T), layout, what=(layout, dtype, T))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("C", [1, 2, 31, 63, 64, 65, 130])
def test_channels(dtype, C):
    for layout in ("bct", "btc"):
        check(make(3, C, 140, dtype, layout, C), layout, state=False, what=(layout, dtype, C))


@pytest.mark.parametrize("layout", ["bct", "btc"])
@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,C,T", [(2, 5, 7), (1, 6, 131), (2, 65, 300), (1, 2, 1100)])
def test_parts_of_a_projection_in_reverse(layout, dtype, B, C, T):
    """x and the gates are chunks of one tensor, the gradients chunks of another, at addresses
    that are aligned to one element."""
    d = make(B, C, T, dtype, layout, 7, packed=True, shift=1)
    dim = 1 if layout == "bct" else 2
    shape = list(d["x"].shape)
    shape[dim] *= 3
    whole = torch.full([torch.Size(shape).numel() + 3], float("nan"), dtype=DT[dtype], device="cuda")
    dproj = whole[1:-2].view(shape)
    grads = dict(zip(("dx", "dr", "di"), dproj.chunk(3, dim=dim)))
    check(d, layout, reverse=True, grads=grads, what=(layout, dtype, B, C, T))
    assert torch.isfinite(dproj).all()
    assert whole[0].isnan() and whole[-2:].isnan().all()  # nothing beside them


@pytest.mark.parametrize("layout", ["bct", "btc"])
@pytest.mark.parametrize("reverse", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "f16"])
@pytest.mark.parametrize("T", [3, 50, 200, 700])
def test_ragged(layout, reverse, dtype, T):
    """Lengths 0, 1, T, between and outside 0..T; NaN in the padding, which is not read."""
    lengths = [T, 0, 1, T // 2, T - 1, -3, T + 9]
    d = make(len(lengths), 3, T, dtype, layout, T)
    for b, n in enumerate(lengths):
        for k in ("x", "r", "i", "dh"):
            t = d[k] if layout == "bct" else d[k].transpose(1, 2)
            t[b, :, max(n, 0):] = float("nan")
    h, out = check(d, layout, lengths=lengths, reverse=reverse, what=(layout, reverse, dtype, T))
    for t in (h, out["dx"], out["dr"], out["di"]):
        t = t if layout == "bct" else t.transpose(1, 2)
        for b, n in enumerate(lengths):
            assert (t[b, :, max(n, 0):] == 0).all()


@pytest.mark.parametrize("layout", ["bct", "btc"])
def test_long_sequences(layout):
    """Many tiles, few rows; exact against fp64 over the whole length."""
    check(make(1, 2, 9001, "f32", layout, 3), layout, what=(layout, 9001))
    check(make(2, 3, 5000, "bf16", layout, 4), layout, reverse=True, lengths=[4999, 2100], what=(layout, 5000))


@pytest.mark.parametrize("layout", ["bct", "btc"])
@pytest.mark.parametrize("reverse", [False, True])
def test_spread_tiles(layout, reverse):
    """Few rows: the tiles of a row lie in several workgroups (4096 positions of a plane, 128 or
    256 of tokens each), in groups of 16; lengths that end in any of them, or before the first."""
    lengths = [9000, 0, 1, 4096, 4097, 8192, 127, 129, 2500]
    d = make(len(lengths), 2, 9000, "f32", layout, 21)
    for b, n in enumerate(lengths):
        for k in ("x", "r", "i", "dh"):
            t = d[k] if layout == "bct" else d[k].transpose(1, 2)
            t[b, :, n:] = float("nan")
    check(d, layout, lengths=lengths, reverse=reverse, what=(layout, reverse, 9000))


@pytest.mark.parametrize("layout,T,dtype", [("bct", 70000, "f32"), ("btc", 4400, "f16")])
def test_past_a_group_of_tiles(layout, T, dtype):
    check(make(1, 3, T, dtype, layout, 22), layout, what=(layout, T, dtype))


def test_planes_of_images():
    d = make(2, 3, 14 * 14, "f32", "bct", 5)
    import aware_conv_amd as A
    h, last, _ = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"])
    q = {k: d[k].view(2, 3, 14, 14) for k in ("x", "r", "i")}
    h4, last4, _ = A.gscan_fwd(q["x"], q["r"], q["i"], d["lam"])
    assert torch.equal(h4.flatten(2), h) and torch.equal(last4, last)


@pytest.mark.parametrize("layout", ["bct", "btc"])
def test_gates_at_their_ends(layout):
    """Gates far open and far shut, infinite ones among them: states stay finite, and a shut
    reset gate holds the state."""
    d = make(2, 6, 40, "f32", layout, 9)
    for k, v in (("r", 200.0), ("i", -200.0)):
        t = d[k] if layout == "bct" else d[k].transpose(1, 2)
        t[0, 0], t[0, 1], t[0, 2], t[0, 3] = v, -v, float("inf"), -float("inf")
    check(d, layout, what=layout)


@pytest.mark.parametrize("layout", ["bct", "btc"])
def test_nothing_to_do(layout):
    import aware_conv_amd as A
    for B, C, T in ((2, 3, 0), (0, 3, 5), (2, 0, 5)):
        d = make(B, C, T, "f32", layout, 1) if B * C * T else None
        shape = (B, C, T) if layout == "bct" else (B, T, C)
        x = torch.zeros(shape, device="cuda")
        lam, h0 = torch.zeros(C, device="cuda"), torch.randn(B, C, device="cuda")
        assert d is None
        h, last, st = A.gscan_fwd(x, x, x, lam, h0=h0, layout=layout, save_states=True)
        assert h.shape == x.shape and torch.equal(last, h0)
        dl = torch.randn(B, C, device="cuda")
        g = A.gscan_bwd(x, x, x, lam, st, x, dh_last=dl, layout=layout)
        assert torch.equal(g["dh0"], dl) and torch.equal(g["dlam"], torch.zeros(C, device="cuda"))


@pytest.mark.parametrize("layout", ["bct", "btc"])
@pytest.mark.parametrize("name", ["x", "r", "i", "lam", "h0"])
def test_gradient_against_differences(layout, name):
    """The kernel's gradient along a random direction, against the change of the fp64 loss:
    central differences of step 1e-4 err by about 1e-8 of the third derivatives, far below the
    fp32 bound of 1e-4 of the terms' magnitudes used here."""
    import aware_conv_amd as A
    B, C, T = 2, 3, 150
    d = make(B, C, T, "f32", layout, 11)
    form = {"layout": layout}
    _, _, st = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"], h0=d["h0"], save_states=True, **form)
    g = A.gscan_bwd(d["x"], d["r"], d["i"], d["lam"], st, d["dh"], dh_last=d["dh_last"], **form)
    a = {k: bct(d[k], layout) if k in "xri" else d[k].double().cpu() for k in ("x", "r", "i", "lam", "h0")}
    dh, dl = bct(d["dh"], layout), d["dh_last"].double().cpu()
    way = torch.randn(a[name].shape, generator=torch.Generator().manual_seed(2), dtype=torch.float64)

    def loss(e):
        b = dict(a)
        b[name] = a[name] + e * way
        h, last, _ = ref.fwd(b["x"], b["r"], b["i"], b["lam"], h0=b["h0"])
        return float((h * dh).sum() + (last * dl).sum())

    slope = (loss(1e-4) - loss(-1e-4)) / 2e-4
    got = g["d" + name]
    terms = (bct(got, layout) if name in "xri" else got.double().cpu()) * way
    assert abs(float(terms.sum()) - slope) <= 1e-4 * float(terms.abs().sum())


def test_autograd():
    """Through the autograd function, with rows that are not adjacent, expanded inputs (whose
    gradient sums over the copies) and gradients of only some inputs."""
    import aware_conv_amd as A
    d = make(2, 4, 60, "f32", "bct", 12)
    x = d["x"].transpose(1, 2).contiguous().transpose(1, 2).requires_grad_()  # [B, C, T], channels adjacent
    r = d["r"][:, :1].detach().clone().requires_grad_()  # one gate for all channels
    lam = d["lam"].clone().requires_grad_()
    h0 = d["h0"][:1].clone().requires_grad_()
    h, last = A.gated_scan(x, r.expand_as(x), d["i"], lam, h0=h0.expand(2, 4))
    ((h * d["dh"]).sum() + (last * d["dh_last"]).sum()).backward()
    a = [t.double().cpu() for t in (d["x"], d["r"][:, :1].expand_as(x), d["i"], d["lam"])]
    w = ref.bwd(*a, d["dh"].double().cpu(), h0=d["h0"][:1].expand(2, 4).double().cpu(),
                dh_last=d["dh_last"].double().cpu())
    close("dx", x.grad, w["dx"])
    close("dlam", lam.grad, w["dlam"], mass=w["mass"])
    close("dr", r.grad, w["dr"].sum(1, keepdim=True))
    close("dh0", h0.grad, w["dh0"].sum(0, keepdim=True))
    # the last state alone
    x2 = d["x"].clone().requires_grad_()
    A.gated_scan(x2, d["r"], d["i"], d["lam"])[1].sum().backward()
    w = ref.bwd(*[t.double().cpu() for t in (d["x"], d["r"], d["i"], d["lam"])],
                torch.zeros(2, 4, 60, dtype=torch.float64), dh_last=torch.ones(2, 4, dtype=torch.float64))
    close("dx", x2.grad, w["dx"])


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,C", [(1, 1), (3, 7), (5, 513), (70, 96)])
def test_step(dtype, B, C):
    """Single positions on a cache: slots in any order, two of them out of range."""
    import aware_conv_amd as A
    print("\ncase step %s" % ((dtype, B, C),), flush=True)
    d = make(B, 3 * C, 1, dtype, "bct", 13, shift=1)
    proj = d["x"].view(B, 3 * C)
    x, r, i = proj.chunk(3, dim=1)
    lam = d["lam"][:C].contiguous()
    S = B + 4
    cache = torch.randn(S, C, generator=torch.Generator().manual_seed(1)).cuda()
    slots = torch.randperm(S, generator=torch.Generator().manual_seed(2))[:B].to(torch.int32)
    if B > 3:
        slots[1], slots[2] = -1, S
    before = cache.clone()
    h = A.gscan_step(x, r, i, lam, cache, slots=slots.cuda())
    on = [(b, int(s)) for b, s in enumerate(slots) if 0 <= s < S]
    want = before.double().cpu().clone()
    wh = torch.zeros(B, C, dtype=torch.float64)
    for b, s in on:
        v, _, _ = ref.fwd(*[t[b:b + 1, :, None].double().cpu() for t in (x, r, i)], lam.double().cpu(),
                          h0=want[s:s + 1])
        wh[b] = want[s] = v[0, :, 0]
    close("h", h, wh)
    close("cache", cache, want)
    used = {s for _, s in on}
    for s in range(S):
        if s not in used:
            assert torch.equal(cache[s], before[s])
    if B <= S:
        c2 = before.clone()
        h2 = A.gscan_step(x, r, i, lam, c2)
        v, _, _ = ref.fwd(*[t[:, :, None].double().cpu() for t in (x, r, i)], lam.double().cpu(),
                          h0=before[:B].double().cpu())
        close("h", h2, v[:, :, 0])
        assert torch.equal(c2[B:], before[B:])


def test_steps_continue_a_scan():
    """A prompt through gscan_fwd, then tokens one by one on its last state, against one scan."""
    import aware_conv_amd as A
    B, C, T = 3, 40, 90
    d = make(B, C, T, "f32", "btc", 14)
    h, last, _ = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"], layout="btc")
    cut = 70
    parts = [d[k][:, :cut] for k in ("x", "r", "i")]
    _, cache, _ = A.gscan_fwd(*parts, d["lam"], layout="btc")
    for t in range(cut, T):
        got = A.gscan_step(d["x"][:, t], d["r"][:, t], d["i"][:, t], d["lam"], cache)
        close("h", got, h[:, t].double().cpu())
    close("last", cache, last.double().cpu())


@pytest.mark.parametrize("layout,B,C,T", [("bct", 2, 3, 1500), ("btc", 2, 70, 600), ("bct", 3, 5, 49)])
def test_graph_and_streams(layout, B, C, T):
    """Captured calls give the eager bits on every replay, and calls on two streams at once give
    those of calls one after the other."""
    import aware_conv_amd as A
    d = make(B, C, T, "f32", layout, 15)
    print("\ncase graph gscan %s" % ((layout, B, C, T),), flush=True)

    def step(ws=None):
        h, last, st = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"], h0=d["h0"], layout=layout,
                                  save_states=True, workspace=ws)
        g = A.gscan_bwd(d["x"], d["r"], d["i"], d["lam"], st, d["dh"], dh_last=d["dh_last"],
                        layout=layout, workspace=ws)
        return [h, last] + [g[n] for n in ("dx", "dr", "di", "dlam", "dh0")]

    want = [t.clone() for t in step()]
    ws = torch.empty(A.gscan.gscan_workspace_size(d["x"], layout) + 16, dtype=torch.uint8, device="cuda")
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ws)
    for _ in range(4):
        for t in out:
            t.fill_(float("nan"))
        ws.fill_(0x5a)
        torch.randn(1 << 18, device="cuda").cumsum(0)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, want))
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            got.append(step())
    torch.cuda.synchronize()
    for run in got:
        assert all(torch.equal(a, b) for a, b in zip(run, want))


def test_a_stream_of_its_own():
    """Calls given a stream: their workspace must not be handed out again, on the current stream,
    while they run."""
    import aware_conv_amd as A
    d = make(2, 70, 3000, "f32", "btc", 16)
    form = {"layout": "btc"}
    h, _, st = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"], save_states=True, **form)
    want = [h] + list(A.gscan_bwd(d["x"], d["r"], d["i"], d["lam"], st, d["dh"], **form).values())
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(5):
        h, _, st = A.gscan_fwd(d["x"], d["r"], d["i"], d["lam"], save_states=True, stream=side, **form)
        g = A.gscan_bwd(d["x"], d["r"], d["i"], d["lam"], st, d["dh"], stream=side, **form)
        # on the current stream, as large as the workspaces were
        junk = [torch.full((1 << 20,), 0x5a, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip([h] + list(g.values()), want))
        del junk


def test_second_derivatives_are_refused():
    import aware_conv_amd as A
    d = make(1, 2, 9, "f32", "bct", 17)
    x = d["x"].clone().requires_grad_()
    h = A.gated_scan(x, d["r"], d["i"], d["lam"])[0]
    g, = torch.autograd.grad(h.square().sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()
