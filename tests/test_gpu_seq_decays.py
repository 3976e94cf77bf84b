"""The recurrence with decays far from the usual, against the formulas in fp64."""
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu


def bct(t, layout):
    t = t.detach().double().cpu()
    return t if layout == "bct" else t.transpose(1, 2)


@pytest.mark.parametrize("layout", ["bct", "btc"])
@pytest.mark.parametrize("T", [30, 300, 9000])
def test_decays_from_none_to_all(layout, T):
    """lam from -60 (a state that 1e26 positions would halve) to 200 (nothing is kept).  Each
    channel by its own largest value: a state that is never forgotten adds up T roundings of
    either sign, sqrt(9000) * 2^-24 = 6e-6 of it, within the 1e-5."""
    import aware_conv_amd as A
    print("\ncase decays %s" % ((layout, T),), flush=True)
    lam = torch.tensor([-60.0, -40.0, -25.0, -17.0, -10.0, -6.0, -3.0, 0.0, 1.0, 4.0, 12.0, 30.0, 88.0, 200.0])
    B, C = 2, len(lam)
    g = torch.Generator().manual_seed(T)
    shape = (B, C, T) if layout == "bct" else (B, T, C)
    d = {k: torch.randn(shape, generator=g) for k in ("x", "r", "i", "dh")}
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
        w = want[n]
        if n == "dlam":
            size = want["mass"]
        else:
            size = w.abs().amax([k for k in range(w.dim()) if k != 1], keepdim=True)
        assert ((u - w).abs() <= 1e-5 * size + 2.0 ** -24 * w.abs() + 1e-37).all(), n
