"""The recurrence in forms that its size selects, and on values at the ends of
what its inputs may hold, against the formulas in fp64.

Tolerances are those of tests/test_gpu_gscan.py (1e-5 of the largest value of
a tensor and half a unit in the last place of the output's type; dlam 1e-5 of
the sum of the magnitudes that it sums)."""
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
TINY = {"f32": 0.0, "f16": 2.0 ** -25, "bf16": 0.0}


def lam_of(a):
    return torch.log(torch.expm1(-torch.log(a.double()) / 8)).float()


# ---------------------------------------------------------------------------
# single positions, four sequences to a thread
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("B,C", [(2049, 1025), (2050, 1024), (4195, 501)])
def test_many_single_positions(dtype, B, C):
    """2^21 elements and more: sequences that do not fill a group of four, odd channels, parts of
    a projection, slots out of range anywhere in a group."""
    import aware_conv_amd as A
    print("\ncase many steps %s" % ((dtype, B, C),), flush=True)
    g = torch.Generator(device="cuda").manual_seed(B)
    x, r, i = torch.randn(B, 3 * C, generator=g, device="cuda").to(DT[dtype]).chunk(3, dim=1)
    lam = lam_of(0.5 + 0.499 * torch.rand(C, generator=g, device="cuda"))
    S = B + 7
    cache = torch.randn(S, C, generator=g, device="cuda")
    slots = torch.randperm(S, generator=g, device="cuda")[:B].to(torch.int32)
    off = torch.zeros(B, dtype=torch.bool, device="cuda")
    off[torch.randint(0, B, (60,), generator=g, device="cuda")] = True
    off[-1] = True
    slots[off] = torch.tensor([-1, S, -2 ** 31, 2 ** 31 - 1], device="cuda").repeat(B)[:B].to(torch.int32)[off]
    for s in (slots, None):
        state = cache.clone()
        h = A.gscan_step(x, r, i, lam, state, slots=s)
        _, a, _, b = ref.gates(x.double(), r.double(), i.double(), lam.double(), 8.0)
        at = torch.arange(B, device="cuda") if s is None else slots.long()
        on = torch.ones_like(off) if s is None else ~off
        want = a * cache.double()[at.clamp(0, S - 1)] + b
        want[~on] = 0
        near = 1e-5 * want.abs().max() + HALF_ULP[dtype] * want.abs() + TINY[dtype]
        assert ((h.double() - want).abs() <= near).all()
        kept = cache.double()
        kept[at[on]] = want[on]
        assert ((state.double() - kept).abs() <= 1e-5 * want.abs().max()).all()
        same = torch.ones(S, dtype=torch.bool, device="cuda")
        same[at[on]] = False
        assert torch.equal(state[same], cache[same])


# ---------------------------------------------------------------------------
# planes whose workgroups take several tiles each
# ---------------------------------------------------------------------------

def scan64(a, b, first):
    """h_t = a_t h_{t-1} + b_t along the last axis, from `first`: pieces side by side, then joined."""
    T = a.shape[-1]
    n = int(T ** 0.5)
    cut = -(-T // n) * n
    a = torch.nn.functional.pad(a, (0, cut - T), value=1.0).unflatten(-1, (n, cut // n)).clone()
    h = torch.nn.functional.pad(b, (0, cut - T)).unflatten(-1, (n, cut // n)).clone()
    for t in range(1, cut // n):
        h[..., t] += a[..., t] * h[..., t - 1]
        a[..., t] *= a[..., t - 1]  # of the piece so far
    for k in range(n):
        h[..., k, :] += a[..., k, :] * first.unsqueeze(-1)
        first = h[..., k, -1]
    return h.flatten(-2)[..., :T]


def formulas(x, r, i, lam, dh, h0, dh_last, lengths, reverse):
    """Outputs and gradients of [B, C, T] inputs in fp64, and the mass of dlam."""
    T = x.shape[-1]
    pos = torch.arange(T, device=x.device)
    n = lengths.view(-1, 1, 1)
    live = (pos < n).expand_as(x)
    order = torch.where(pos < n, n - 1 - pos if reverse else pos.view(1, 1, -1), pos).expand_as(x)
    x, r, i, dh = (torch.where(live, t.double(), 0.0).gather(2, order) for t in (x, r, i, dh))
    l3 = lam.double()[None, :, None]
    L, a, w, b = ref.gates(x, r, i, l3, 8.0)
    held = torch.where(live, a, 1.0)
    h = scan64(held, torch.where(live, b, 0.0), h0.double())
    before = torch.cat([h0.double().unsqueeze(-1), h[..., :-1]], -1)
    # u_t = a_t (dh_t + u_{t+1})
    u = scan64(held.flip(-1), (held * dh).flip(-1), dh_last.double()).flip(-1)
    g = dh + torch.cat([u[..., 1:], dh_last.double().unsqueeze(-1)], -1)
    si = ref.sig(i)
    d = g * (a * before - si * x * a * a / w)
    e = torch.where(live, -d * ref.sig(r), 0.0)
    k = 8 * ref.sig(lam.double())
    out = {"h": h, "dx": g * w * si, "dr": d * L * ref.sig(-r), "di": g * w * si * x * ref.sig(-i)}
    out = {m: torch.where(live, t, 0.0).gather(2, order) for m, t in out.items()}
    return dict(out, h_last=h[..., -1], dh0=u[..., 0], dlam=k * e.sum((0, 2)), mass=k * e.abs().sum((0, 2)))


@pytest.mark.parametrize("dtype,reverse", [("f32", False), ("f32", True), ("bf16", True), ("f16", False)])
def test_shares_of_several_tiles(dtype, reverse):
    """766 rows of 18 tiles: 13788 units, three to a workgroup, the last share short; lengths that
    end in any tile, so that padded and valid ones follow one another in a share; more than a group
    of 16 tiles."""
    import aware_conv_amd as A
    print("\ncase shares %s" % ((dtype, reverse),), flush=True)
    B, C, T = 383, 2, 70001
    g = torch.Generator(device="cuda").manual_seed(9)
    x, r, i, dh = (torch.randn(B, C, T, generator=g, device="cuda").to(DT[dtype]) for _ in range(4))
    lengths = torch.randint(0, T + 1, (B,), generator=g, device="cuda").to(torch.int32)
    lengths[:9] = torch.tensor([T, 0, 1, T - 1, 4096, 4097, 65536, 65537, 69633], device="cuda")
    pad = torch.arange(T, device="cuda") >= lengths.view(-1, 1, 1)
    for t in (x, r, i, dh):
        t.masked_fill_(pad, float("nan"))
    lam = lam_of(0.5 + 0.499 * torch.rand(C, generator=g, device="cuda"))
    h0, dh_last = torch.randn(B, C, generator=g, device="cuda"), torch.randn(B, C, generator=g, device="cuda")
    form = {"lengths": lengths, "reverse": reverse}
    h, h_last, states = A.gscan_fwd(x, r, i, lam, h0=h0, save_states=True, **form)
    got = dict(A.gscan_bwd(x, r, i, lam, states, dh, dh_last=dh_last, **form), h=h, h_last=h_last)
    want = formulas(x, r, i, lam, dh, h0, dh_last, lengths, reverse)
    for n in ("h", "dx", "dr", "di", "h_last", "dh0"):
        a, b = got[n].double(), want[n]
        half, tiny = (HALF_ULP[dtype], TINY[dtype]) if a.dim() == 3 else (2.0 ** -24, 0.0)
        assert ((a - b).abs() <= 1e-5 * b.abs().max() + half * b.abs() + tiny).all(), n
        if a.dim() == 3:
            assert (a.masked_select(pad) == 0).all(), n
    assert ((got["dlam"].double() - want["dlam"]).abs() <= 1e-5 * want["mass"] + 2.0 ** -24 * want["dlam"].abs()).all()


# ---------------------------------------------------------------------------
# values that are not finite
# ---------------------------------------------------------------------------

def bct(t, layout):
    t = t.detach().double().cpu()
    return t if layout == "bct" else t.transpose(1, 2)


ONES = torch.tensor([-1], dtype=torch.int32).view(torch.float32)  # the NaN of all ones


@pytest.mark.parametrize("layout", ["bct", "btc"])
@pytest.mark.parametrize("T", [5, 100, 700, 9000])
@pytest.mark.parametrize("name,value", [("x", float("inf")), ("x", float("nan")), ("r", float("nan")),
                                        ("dh", float("nan")), ("all", None)])
def test_what_is_not_finite_goes_where_the_formula_takes_it(layout, T, name, value):
    """One position of one row; the others, and what does not depend on it, keep their values.  A
    NaN of all ones passes between workgroups, whose words mean "not there" by that pattern."""
    import aware_conv_amd as A
    print("\ncase not finite %s" % ((layout, T, name, value),), flush=True)
    B, C = 2, 3
    g = torch.Generator().manual_seed(T)
    shape = (B, C, T) if layout == "bct" else (B, T, C)
    d = {k: torch.randn(shape, generator=g) for k in ("x", "r", "i", "dh")}
    for k, t in d.items():
        if name in (k, "all"):
            (t if layout == "bct" else t.transpose(1, 2))[1, 1, T // 3] = ONES[0] if value is None else value
    lam = lam_of(0.5 + 0.499 * torch.rand(C, generator=g))
    h0, dh_last = torch.randn(B, C, generator=g), torch.randn(B, C, generator=g)
    q = {k: t.cuda() for k, t in d.items()}
    h, h_last, states = A.gscan_fwd(q["x"], q["r"], q["i"], lam.cuda(), h0=h0.cuda(), layout=layout, save_states=True)
    got = dict(A.gscan_bwd(q["x"], q["r"], q["i"], lam.cuda(), states, q["dh"], dh_last=dh_last.cuda(), layout=layout),
               h=h, h_last=h_last)
    a = [bct(d[k], layout) for k in ("x", "r", "i")] + [lam.double()]
    wh, wl, _ = ref.fwd(*a, h0=h0.double())
    want = dict(ref.bwd(*a, bct(d["dh"], layout), h0=h0.double(), dh_last=dh_last.double()), h=wh, h_last=wl)
    for n in ("h", "dx", "dr", "di", "h_last", "dh0", "dlam"):
        u = bct(got[n], layout) if got[n].dim() == 3 else got[n].double().cpu()
        fine = torch.isfinite(want[n])
        assert torch.equal(torch.isfinite(u), fine), n
        size = want["mass"][fine] if n == "dlam" else want[n][fine].abs().max()
        assert ((u - want[n])[fine].abs() <= 1e-5 * size + 2.0 ** -24 * want[n][fine].abs()).all(), n
