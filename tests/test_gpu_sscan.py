"""The selective scan on the GPU against its formulas in fp64.

Tolerances.  A decay is formed to a few units of 2^-24, and a state adds such an error at each
step and forgets it with the decay: at most 0.999 here, about 1000 steps, errors of either sign,
so about sqrt(500) * 2 * 6e-8 = 3e-6 of the states' size.  Every output is a sum of products with
states, or with gradients that go back in the same way: 1e-5 of the largest sum of its terms'
magnitudes.  16-bit outputs add half a unit in their last place."""
import pytest
import torch

import token_reference as ref

pytestmark = pytest.mark.gpu

HALF_ULP = {torch.float32: 2.0 ** -24, torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}
TINY = {torch.float32: 0.0, torch.float16: 2.0 ** -25, torch.bfloat16: 0.0}
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
WIDE, LOW = ("x", "dt", "z", "dy"), ("b", "c")


def close(name, got, want, mass=None):
    got, dt = got.detach().double().cpu(), got.dtype
    assert got.shape == want.shape, name
    top = float((want.abs() if mass is None else mass).max()) if want.numel() else 0.0
    bound = 1e-5 * top + HALF_ULP[dt] * want.abs() + TINY[dt]
    assert torch.isfinite(got).all(), name
    err = (got - want).abs()
    assert (err <= bound).all(), "%s: error %.3g, largest sum of magnitudes %.3g" % (name, float(err.max()), top)


def place(t, shift=0):
    """`t` on the GPU, `shift` elements off its allocation."""
    flat = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
    flat[shift:] = t.flatten().cuda()
    return flat[shift:].view(t.shape)


def make(B, T, D, N, G=1, dtype="f32", seed=0, without=(), packed=False, shift=0):
    """What a scan and its gradients take; `without` are left out."""
    g = torch.Generator().manual_seed(seed)
    dt = DT[dtype]
    rand = lambda *n: torch.randn(*n, generator=g)  # noqa: E731
    s = {k: rand(B, T, D).to(dt) for k in WIDE}
    s.update({k: rand(B, T, G * N).to(dt) for k in LOW})
    if packed:  # x and z are halves of one projection; b and c parts of another
        s["x"], s["z"] = place(torch.cat([s["x"], s["z"]], 2), shift).chunk(2, dim=2)
        s["b"], s["c"] = place(torch.cat([rand(B, T, 5).to(dt), s["b"], s["c"]], 2), shift)[..., 5:].chunk(2, dim=2)
    s = {k: t if t.is_cuda else place(t, shift) for k, t in s.items()}
    # steps of 0.001 to 0.1 and decay rates of 1 to N
    step = 10 ** (-3 + 2 * torch.rand(D, generator=g, dtype=torch.float64))
    s["dt_bias"] = torch.log(torch.expm1(step)).float().cuda()
    s["a_log"] = (torch.arange(1, N + 1).log().repeat(D, 1) + 0.1 * rand(D, N)).cuda()
    s["d"] = rand(D).cuda()
    s["h0"], s["dh_last"] = rand(B, D, N).cuda(), rand(B, D, N).cuda()
    for k in without:
        s[k] = None
    return s


def wide64(t):
    return None if t is None else t.detach().double().cpu()


def check(s, lengths=None, what=""):
    import aware_conv_amd as A
    print("\ncase sscan %s" % (what,), flush=True)
    form = {k: s[k] for k in ("d", "z", "dt_bias")}
    form["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    args = [s[k] for k in ("x", "dt", "a_log", "b", "c")]
    y, h_last, states = A.sscan_fwd(*args, h0=s["h0"], save_states=True, **form)
    plain = A.sscan_fwd(*args, h0=s["h0"], **form)
    g = A.sscan_bwd(*args, states, s["dy"], dh_last=s["dh_last"], **form)
    torch.cuda.synchronize()
    assert plain[2] is None and torch.equal(plain[0], y) and torch.equal(plain[1], h_last)
    r = {k: wide64(s[k]) for k in s}
    if lengths is not None:  # what lies beyond the lengths is not read
        for i, n in enumerate(ref.counts(*s["x"].shape[:2], lengths)):
            for k in WIDE + LOW:
                if r[k] is not None:
                    r[k][i, n:] = 0
    want, mass = ref.sscan(lengths=lengths, **r)
    close("y", y, want["y"], mass["y"])
    close("h_last", h_last, want["h_last"])
    for k in ("dx", "ddt", "db", "dc", "da_log", "dd", "dz", "ddt_bias", "dh0"):
        term = {"dd": "d", "dz": "z", "ddt_bias": "dt_bias"}.get(k)
        if term and s[term] is None:
            assert g[k] is None
        else:
            close(k, g[k], want[k], mass.get(k))
    return y, h_last, g


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [1, 2, 3, 4, 5, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 129, 257])
def test_lengths(dtype, T):
    check(make(2, T, 5, 6, dtype=dtype, seed=T), what=(dtype, T))


@pytest.mark.parametrize("N", [1, 2, 3, 4, 5, 7, 8, 9, 12, 15, 16, 17, 21, 31, 32, 33, 48, 63, 64])
def test_states(N):
    for T in (40, 260):
        check(make(2, T, 18, N, dtype="f32", seed=N), what=("states", N, T))
    check(make(1, 70, 18, N, dtype="bf16", seed=N), what=("states", N, "bf16"))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("D,G", [(1, 1), (15, 1), (16, 1), (17, 1), (63, 1), (64, 1), (65, 1), (130, 1), (130, 2),
                                 (66, 3), (12, 12), (192, 4)])
def test_channels(dtype, D, G):
    check(make(2, 37, D, 4, G=G, dtype=dtype, seed=D + G), what=(dtype, D, G))


@pytest.mark.parametrize("without", [(), ("z",), ("d",), ("dt_bias",), ("h0",), ("dh_last",), ("z", "d"),
                                     ("z", "d", "dt_bias", "h0", "dh_last")])
def test_absent_terms(without):
    s = make(2, 50, 20, 16, dtype="f32", seed=3, without=without)
    if s["dt_bias"] is None:
        s["dt"] -= 4
    check(s, what=without)


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T", [40, 700])
def test_ragged(dtype, T):
    """Lengths of zero, one, the ends of tiles, beyond T and below 0; NaN where nothing is read."""
    lengths = [T, 0, 1, 16, 17, 31, 32, 33, -5, T + 9, T - 1]
    s = make(len(lengths), T, 7, 5, dtype=dtype, seed=T)
    for i, n in enumerate(ref.counts(len(lengths), T, lengths)):
        for k in WIDE + LOW:
            s[k][i, n:] = float("nan")
    y, _, g = check(s, lengths, what=("ragged", dtype, T))
    for i, n in enumerate(ref.counts(len(lengths), T, lengths)):
        for t in (y, g["dx"], g["ddt"], g["dz"], g["db"], g["dc"]):
            assert (t[i, n:] == 0).all()


def test_all_empty():
    s = make(3, 40, 7, 5, seed=1)
    check(s, [0, 0, 0], what="all empty")


@pytest.mark.parametrize("B,T,D,N", [(1, 5000, 8, 16), (3, 1111, 70, 16), (1, 2100, 20, 4), (2, 900, 17, 40)])
def test_segments(B, T, D, N):
    """Few channels and long sequences: several segments of a sequence run at once."""
    check(make(B, T, D, N, dtype="f32", seed=T), what=("segments", B, T, D, N))
    check(make(B, T, D, N, dtype="f32", seed=T), [T // 3] * B, what=("segments, ragged", B, T, D, N))


def test_many_sequences():
    check(make(130, 33, 130, 3, dtype="bf16", seed=4), what="many sequences")


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("shift", [0, 1, 3])
def test_views(dtype, shift):
    """Parts of projections, at odd addresses; gradients written as parts too."""
    import aware_conv_amd as A
    s = make(2, 45, 19, 16, dtype=dtype, seed=shift, packed=True, shift=shift)
    y, _, g = check(s, what=("views", dtype, shift))
    wide = place(torch.full((2, 45, 2 * 19), 7.0, dtype=DT[dtype]), shift)
    low = place(torch.full((2, 45, 5 + 32), 7.0, dtype=DT[dtype]), shift)
    dx, dz = wide.chunk(2, dim=2)
    grads = {"dx": dx, "dz": dz, "db": low[..., 5:21], "dc": low[..., 21:]}
    args = [s[k] for k in ("x", "dt", "a_log", "b", "c")]
    form = {k: s[k] for k in ("d", "z", "dt_bias")}
    states = A.sscan_fwd(*args, h0=s["h0"], save_states=True, **form)[2]
    again = A.sscan_bwd(*args, states, s["dy"], dh_last=s["dh_last"], grads=grads, **form)
    for k in g:
        assert torch.equal(again[k], g[k]), k
    assert (low[..., :5] == 7).all() and again["dx"] is dx


def test_broadcast_inputs():
    """One sequence's b and c for the whole batch."""
    s = make(3, 40, 18, 8, seed=9)
    for k in LOW:
        s[k] = s[k][:1].expand(3, -1, -1)
    check(s, what="broadcast")


def test_offsets_beyond_32_bits():
    import aware_conv_amd as A
    s = make(2, 50, 33, 4, dtype="bf16", seed=2)
    want = A.sscan_fwd(*[s[k] for k in ("x", "dt", "a_log", "b", "c")], z=s["z"])[:2]
    far = torch.zeros((1 << 31) + 50 * 40, dtype=torch.bfloat16, device="cuda").as_strided((2, 50, 33), (1 << 31, 40, 1))
    far.copy_(s["x"])
    rows = torch.zeros(50 * (1 << 26), dtype=torch.bfloat16, device="cuda").as_strided((2, 50, 33), (64, 1 << 26, 1))
    rows.copy_(s["z"])
    y = torch.zeros((1 << 31) + 50 * 40, dtype=torch.bfloat16, device="cuda").as_strided((2, 50, 33), (1 << 31, 40, 1))
    got = A.sscan_fwd(far, s["dt"], s["a_log"], s["b"], s["c"], z=rows, y=y)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and got[0] is y


def test_slow_decays():
    """A state that lasts 100000 positions: the hardware's power is not exact near 1, and its error
    would add up (1e-5 of the size here; the uncorrected power was 6e-5 off)."""
    import aware_conv_amd as A
    T = 20000
    s = make(1, T, 16, 4, seed=5)
    s["dt"] = torch.zeros_like(s["dt"])
    s["dt_bias"] = torch.log(torch.expm1(torch.logspace(-5, -2, 16, dtype=torch.float64))).float().cuda()
    s["a_log"] = torch.zeros(16, 4, device="cuda")
    s["h0"].fill_(1.0)
    s["x"] = torch.full_like(s["x"], 0.25)
    s["b"] = torch.full_like(s["b"], 0.5)
    r = {k: wide64(v) for k, v in s.items()}
    r["dy"] = r["dh_last"] = None
    want, _ = ref.sscan(**r)
    h = A.sscan_fwd(s["x"], s["dt"], s["a_log"], s["b"], s["c"], h0=s["h0"], dt_bias=s["dt_bias"])[1]
    assert ((h.double().cpu() - want["h_last"]).abs() <= 1e-5 * want["h_last"].abs()).all()


def test_steps_of_any_size():
    """dt from where softplus is 1e-30 to where it is the value itself, rates from 1e-6 to 1e6."""
    s = make(1, 64, 16, 8, seed=6, without=("dt_bias",))
    s["dt"] = torch.linspace(-70, 60, 64 * 16, device="cuda").view(1, 64, 16)[:, torch.randperm(64)]
    s["a_log"] = torch.linspace(-14, 14, 16 * 8, device="cuda").view(16, 8)
    check(s, what="any size")


@pytest.mark.parametrize("lengths", [None, [37, 5, 0]])
def test_rates_beyond_the_largest_number(lengths):
    """exp(a_log) is infinite: such a state forgets everything at each step, and what is behind a
    sequence leaves it as it is."""
    import aware_conv_amd as A
    s = make(3, 37, 18, 8, seed=6)
    s["a_log"][:, 3] = 100.0
    form = {k: s[k] for k in ("d", "z", "dt_bias")}
    form["lengths"] = None if lengths is None else torch.tensor(lengths, dtype=torch.int32, device="cuda")
    args = [s[k] for k in ("x", "dt", "a_log", "b", "c")]
    y, h, states = A.sscan_fwd(*args, h0=s["h0"], save_states=True, **form)
    g = A.sscan_bwd(*args, states, s["dy"], dh_last=s["dh_last"], **form)
    for i, n in enumerate(ref.counts(3, 37, lengths)):
        if n:  # the last step's input alone
            t = n - 1
            u = torch.nn.functional.softplus(s["dt"][i, t] + s["dt_bias"]) * s["x"][i, t]
            assert (h[i, :, 3] - u * s["b"][i, t, 3]).abs().max() <= 1e-6 * h.abs().max()
        else:
            assert torch.equal(h[i], s["h0"][i])
    assert torch.isfinite(y).all() and torch.isfinite(h).all()
    for k in ("dx", "ddt", "dz", "db", "dc", "dd", "ddt_bias", "dh0", "da_log"):
        assert torch.isfinite(g[k]).all(), k


def test_no_channels():
    """Sums over no channels are zero."""
    import aware_conv_amd as A
    z = lambda *n: torch.zeros(*n, device="cuda")  # noqa: E731
    args = [z(2, 20, 0), z(2, 20, 0), z(0, 4), torch.randn(2, 20, 4, device="cuda"), torch.randn(2, 20, 4, device="cuda")]
    y, h, states = A.sscan_fwd(*args, save_states=True)
    low = torch.full((2, 20, 8), 7.0, device="cuda")
    g = A.sscan_bwd(*args, states, y, grads={"db": low[..., :4], "dc": low[..., 4:]})
    assert y.shape == (2, 20, 0) and h.shape == (2, 0, 4) and (low == 0).all() and g["da_log"].shape == (0, 4)


def test_no_positions():
    import aware_conv_amd as A
    s = make(2, 0, 6, 4, seed=1)
    args = [s[k] for k in ("x", "dt", "a_log", "b", "c")]
    y, h, states = A.sscan_fwd(*args, h0=s["h0"], save_states=True)
    g = A.sscan_bwd(*args, states, s["dy"], dh_last=s["dh_last"])
    assert y.shape == (2, 0, 6) and torch.equal(h, s["h0"]) and torch.equal(g["dh0"], s["dh_last"])
    assert (g["da_log"] == 0).all() and g["db"].shape == (2, 0, 4)


def test_two_runs_agree_bit_for_bit():
    s = make(3, 900, 70, 16, dtype="bf16", seed=8)
    a, b = check(s, what="first"), check(s, what="second")
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    for k in a[2]:
        assert torch.equal(a[2][k], b[2][k]), k


@pytest.mark.parametrize("D,T", [(70, 100), (8, 900)])
def test_captured_calls(D, T):
    """Replays, with other inputs and other work between them, give what eager calls give."""
    import aware_conv_amd as A
    s = make(2, T, D, 16, dtype="bf16", seed=D)
    args = [s[k] for k in ("x", "dt", "a_log", "b", "c")]
    form = {k: s[k] for k in ("d", "z", "dt_bias")}

    def run():
        y, h, states = A.sscan_fwd(*args, h0=s["h0"], save_states=True, **form)
        return y, h, A.sscan_bwd(*args, states, s["dy"], dh_last=s["dh_last"], **form)

    run()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        kept = run()
    for k in range(4):
        for n in ("x", "dt", "b", "c", "z", "dy"):
            s[n].copy_(torch.randn(s[n].shape, device="cuda"))
        y, h, g = run()
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(kept[0], y) and torch.equal(kept[1], h), k
        for n in g:
            assert torch.equal(kept[2][n], g[n]), (k, n)


def test_streams():
    import aware_conv_amd as A
    s = make(2, 900, 8, 16, seed=1)
    args = [s[k] for k in ("x", "dt", "a_log", "b", "c")]
    want = A.sscan_fwd(*args, z=s["z"])
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [A.sscan_fwd(*args, z=s["z"], stream=q) for q in streams for _ in range(3)]
    torch.cuda.synchronize()
    for r in got:
        assert torch.equal(r[0], want[0]) and torch.equal(r[1], want[1])


# single positions ------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,D,N,G", [(1, 1, 1, 1), (3, 17, 4, 1), (2, 70, 16, 2), (5, 33, 21, 3), (70, 130, 8, 1),
                                     (2, 12, 64, 12), (1, 384, 16, 1)])
def test_step(dtype, B, D, N, G):
    import aware_conv_amd as A
    print("\ncase sscan step %s" % ((dtype, B, D, N, G),), flush=True)
    s = make(B, 1, D, N, G=G, dtype=dtype, seed=D)
    S = B + 3
    cache = torch.randn(S, D, N, device="cuda")
    before = cache.clone()
    slots = torch.randperm(S)[:B].to(torch.int32)
    if B > 2:
        slots[1], slots[2] = -1, S  # passed over
    on = [i for i in range(B) if 0 <= slots[i] < S]
    form = {"d": s["d"], "dt_bias": s["dt_bias"], "slots": slots.cuda()}
    args = [s["x"][:, 0], s["dt"][:, 0], s["a_log"], s["b"][:, 0], s["c"][:, 0]]
    y = A.sscan_step(*args, cache, z=s["z"][:, 0], **form)
    r = {k: wide64(s[k]) for k in s}
    r["dy"] = r["dh_last"] = None
    r["h0"] = before.double().cpu()[slots.long().clamp(0, S - 1)]
    want, mass = ref.sscan(**r)
    close("y", y[on], want["y"][on, 0], mass["y"][on, 0])
    close("state", cache[slots.long()[on].cuda()], want["h_last"][on])
    rest = [k for k in range(S) if k not in [int(slots[i]) for i in on]]
    assert torch.equal(cache[rest], before[rest])
    off = [i for i in range(B) if i not in on]
    assert (y[off] == 0).all()


def test_step_absent_terms():
    import aware_conv_amd as A
    s = make(4, 1, 20, 16, seed=2)
    args = [s["x"][:, 0], s["dt"][:, 0] - 3, s["a_log"], s["b"][:, 0], s["c"][:, 0]]
    cache = s["h0"].clone()
    y = A.sscan_step(*args, cache)
    r = {k: wide64(s[k]) for k in ("x", "dt", "a_log", "b", "c", "h0")}
    r["dt"] = wide64(args[1])[:, None]
    want, mass = ref.sscan(**r)
    close("y", y, want["y"][:, 0], mass["y"][:, 0])
    close("state", cache, want["h_last"])


@pytest.mark.parametrize("N", [16, 5])
def test_positions_one_by_one(N):
    """A prompt at once and single positions after it give what one pass gives: the same formula in
    two groupings, 1e-5 of the largest."""
    import aware_conv_amd as A
    s = make(3, 60, 40, N, seed=N)
    form = {"d": s["d"], "dt_bias": s["dt_bias"]}
    args = lambda at: [s["x"][:, at], s["dt"][:, at], s["a_log"], s["b"][:, at], s["c"][:, at]]  # noqa: E731
    whole, last, _ = A.sscan_fwd(*args(slice(None)), z=s["z"], h0=s["h0"], **form)
    y, cache, _ = A.sscan_fwd(*args(slice(0, 37)), z=s["z"][:, :37], h0=s["h0"], **form)
    parts = [y] + [A.sscan_step(*args(t), cache, z=s["z"][:, t], **form)[:, None] for t in range(37, 60)]
    assert (torch.cat(parts, 1) - whole).abs().max() <= 1e-5 * whole.abs().max()
    assert (cache - last).abs().max() <= 1e-5 * last.abs().max()


@pytest.mark.parametrize("B,D,N", [(40, 2100, 16), (9, 33000, 5), (33, 33000, 5), (35, 33000, 16)])
def test_many_single_positions(B, D, N):
    """Up to so many that a thread takes two sequences (from 16384 workgroups on); the last pair is not whole."""
    import aware_conv_amd as A
    s = make(B, 1, D, N, dtype="bf16", seed=D)
    S = B + 2
    cache = torch.randn(S, D, N, device="cuda")
    before = cache.clone()
    slots = torch.randperm(S)[:B].to(torch.int32)
    slots[3], slots[B - 1] = S, -7
    form = {"d": s["d"], "dt_bias": s["dt_bias"]}
    at = lambda t, i: t[i:i + 1, 0]  # noqa: E731
    y = A.sscan_step(s["x"][:, 0], s["dt"][:, 0], s["a_log"], s["b"][:, 0], s["c"][:, 0], cache, z=s["z"][:, 0],
                     slots=slots.cuda(), **form)
    for i in range(B):
        k = int(slots[i])
        if not 0 <= k < S:
            assert (y[i] == 0).all()
            continue
        one = before[k:k + 1].clone()
        want = A.sscan_step(at(s["x"], i), at(s["dt"], i), s["a_log"], at(s["b"], i), at(s["c"], i), one, z=at(s["z"], i), **form)
        assert torch.equal(y[i:i + 1], want) and torch.equal(cache[k], one[0])
    rest = [k for k in range(S) if k not in slots.tolist()]
    assert torch.equal(cache[rest], before[rest])


# autograd ----------------------------------------------------------------------

def leaves(s):
    names = [k for k in ("x", "dt", "a_log", "b", "c", "d", "z", "dt_bias", "h0") if s[k] is not None]
    return {k: s[k].detach().clone().requires_grad_() for k in names}


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("use", ["both", "y", "h_last"])
def test_autograd(dtype, use):
    import aware_conv_amd as A
    s = make(2, 50, 20, 16, dtype=dtype, seed=7)
    p = leaves(s)
    y, h = A.selective_scan(**p)
    loss = 0
    if use != "h_last":
        loss = loss + (y * s["dy"]).float().sum()
    if use != "y":
        loss = loss + (h * s["dh_last"]).sum()
    loss.backward()
    r = {k: wide64(s[k]) for k in s}
    if use == "h_last":
        r["dy"] = torch.zeros_like(r["dy"])
    if use == "y":
        r["dh_last"] = None
    want, mass = ref.sscan(**r)
    for k, t in p.items():
        close(k, t.grad, want["d" + k], mass.get("d" + k))


def test_autograd_of_one_input():
    import aware_conv_amd as A
    s = make(1, 20, 6, 4, seed=1)
    b = s["b"].clone().requires_grad_()
    y, _ = A.selective_scan(s["x"], s["dt"], s["a_log"], b, s["c"])
    y.sum().backward()
    assert b.grad is not None
    with torch.no_grad():
        assert not A.selective_scan(s["x"], s["dt"], s["a_log"], b, s["c"])[0].requires_grad


def test_second_derivatives_are_refused():
    import aware_conv_amd as A
    s = make(1, 20, 6, 4, seed=1)
    x = s["x"].clone().requires_grad_()
    y, _ = A.selective_scan(x, s["dt"], s["a_log"], s["b"], s["c"])
    g, = torch.autograd.grad(y.sum(), x, create_graph=True)
    with pytest.raises(RuntimeError):
        g.sum().backward()


def test_gradients_against_differences():
    """Along a random direction, of a loss summed in fp64.  With a step of 2^-7 the difference's own
    error is of order step^2 = 6e-5 and, from outputs of 2^-24, 1e-5: 1e-3 of the loss's terms."""
    import aware_conv_amd as A
    s = make(2, 40, 18, 8, seed=11)
    p = leaves(s)
    y, h = A.selective_scan(**p)
    ((y * s["dy"]).sum() + (h * s["dh_last"]).sum()).backward()

    def loss(q):
        y, h = A.selective_scan(**q)
        return float((y.double() * s["dy"].double()).sum() + (h.double() * s["dh_last"].double()).sum())

    y = y.detach()
    size = float((y.double() * s["dy"].double()).abs().sum() + (h.detach().double() * s["dh_last"].double()).abs().sum())
    for k in p:
        torch.manual_seed(1)
        way = torch.randn_like(p[k])
        at = {n: t.detach() for n, t in p.items()}
        up, down = (loss({**at, k: at[k] + sign * 2 ** -7 * way}) for sign in (1, -1))
        slope = float((p[k].grad.double() * way.double()).sum())
        assert abs((up - down) * 2 ** 6 - slope) <= 1e-3 * size, k


@pytest.mark.parametrize("B", [1 << 25, (1 << 25) - 3])
def test_most_single_positions(B):
    """More sequences than one launch has threads for; one channel of one state, fp32.  Tolerance: h
    takes four roundings, a power to 2 units and softplus to 4 of its last place; y two more."""
    import aware_conv_amd as A
    g = torch.Generator(device="cuda").manual_seed(5)
    r = lambda *s: torch.randn(*s, generator=g, device="cuda")  # noqa: E731
    x, dt, b, c, cache = r(B, 1), r(B, 1), r(B, 1), r(B, 1), r(B, 1, 1)
    a_log = torch.zeros(1, 1, device="cuda")
    before = cache.clone()
    y = A.sscan_step(x, dt, a_log, b, c, cache)
    for part in (slice(0, 1 << 16), slice((1 << 24) - 1000, (1 << 24) + 1000), slice(B - (1 << 16), B)):
        x_, dt_, b_, c_, h_ = (t[part].reshape(-1).double() for t in (x, dt, b, c, before))
        delta = torch.nn.functional.softplus(dt_)
        u = torch.exp(-delta) * h_
        h = u + delta * x_ * b_
        mass = u.abs() * (1 + delta) + (delta * x_ * b_).abs()
        assert ((cache[part].reshape(-1).double() - h).abs() <= 12 * 2.0 ** -23 * mass + 1e-30).all()
        assert ((y[part].reshape(-1).double() - c_ * h).abs() <= 14 * 2.0 ** -23 * (c_.abs() * mass) + 1e-30).all()
