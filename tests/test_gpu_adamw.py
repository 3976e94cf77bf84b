"""The AdamW step on the GPU against its formula in fp64.

Tolerances.  fp32 states are formed by two roundings: 4e-7 of the larger of
their two terms.  A parameter moves by lr * (an expression formed to about 1e-6
of itself) and is rounded once: 2e-7 of itself and 2e-6 of lr * its update.
8-bit states: the code that the definition gives, wherever fp64 and fp32 cannot
differ over it."""
import numpy as np
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu

DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HALF_ULP = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}
HYPER = {"lr": 3e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1}


def place(t, shift):
    flat = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
    flat[shift:] = t.cuda()
    return flat[shift:]


def make(sizes, dtype, bits, master, seed=0, shift=0):
    g = torch.Generator().manual_seed(seed)
    s = {"p": [], "g": [], "m": [], "v": [], "w": [], "ms": [], "vs": []}
    for n in sizes:
        w = torch.randn(n, generator=g) * 0.1
        s["p"].append(place(w.to(DT[dtype]), shift))
        s["w"].append(place(w, shift))
        s["g"].append(place((torch.randn(n, generator=g) * 1e-2).to(DT[dtype]), shift))
        m, v = torch.randn(n, generator=g) * 1e-2, (torch.randn(n, generator=g) * 1e-2) ** 2
        if bits == 8:
            codes = torch.randint(0, 127, (2, n), generator=g, dtype=torch.uint8)
            codes[0] |= (torch.rand(n, generator=g) < 0.5).to(torch.uint8) * 128
            s["m"].append(place(codes[0], shift).view(torch.float8_e4m3fn))
            s["v"].append(place(codes[1], shift).view(torch.float8_e4m3fn))
            for k in ("ms", "vs"):
                s[k].append(place(torch.rand(-(-n // 256), generator=g) * 1e-4, shift))
        else:
            s["m"].append(place(m, shift))
            s["v"].append(place(v, shift))
    if not master:
        s["w"] = None
    if bits == 32:
        s["ms"] = s["vs"] = None
    return s


def arrays(ts):
    return [t.double().cpu().numpy().copy() for t in ts]


def held(codes, scales):
    return [c.float().double().cpu().numpy() * np.repeat(k.double().cpu().numpy(), 256)[:c.numel()]
            for c, k in zip(codes, scales)]


def check(s, dtype, bits, t0=4, clip=None, grad_scale=1.0, what=""):
    import aware_conv_amd as A
    print("\ncase adamw %s" % (what,), flush=True)
    step = torch.full((1,), t0, dtype=torch.int32, device="cuda")
    p0 = arrays(s["w"] or s["p"])
    grads = [g * grad_scale for g in arrays(s["g"])]
    if bits == 8:
        m0, v0 = held(s["m"], s["ms"]), [v ** 2 for v in held(s["v"], s["vs"])]
    else:
        m0, v0 = arrays(s["m"]), arrays(s["v"])
    norm = None
    if clip:
        norm = A.adamw_grad_norm(s["g"], grad_scale=grad_scale)
        want = ref.norm(grads)
        assert abs(float(norm) - want) <= 2.0 ** -23 * want
        # the step's factor goes by the fp32 norm that it is given
        grads = [g * min(1.0, clip / (float(norm) + 1e-6)) for g in grads]
    A.adamw_step(s["p"], s["g"], s["m"], s["v"], step, masters=s["w"], grad_scale=grad_scale,
                 scales=(s["ms"], s["vs"]) if bits == 8 else None, grad_norm=norm, max_norm=clip, **HYPER)
    torch.cuda.synchronize()
    t = t0 + 1
    assert int(step) == t
    off = 0
    for k in range(len(p0)):
        p, m, v = ref.adamw(p0[k], grads[k], m0[k], v0[k], t, **HYPER)
        got = (s["w"] or s["p"])[k].double().cpu().numpy()
        bound = 2e-7 * np.abs(p0[k]) + 2e-6 * np.abs(p - p0[k] * (1 - HYPER["lr"] * HYPER["weight_decay"]))
        if not s["w"]:
            bound = bound + HALF_ULP[dtype] * np.abs(p) + (2.0 ** -25 if dtype == "f16" else 0)
        assert (np.abs(got - p) <= bound).all(), ("p", k)
        if s["w"]:
            assert torch.equal(s["p"][k], s["w"][k].to(s["p"][k].dtype))
        if bits == 32:
            size = np.abs(m0[k]) + np.abs(grads[k])
            assert (np.abs(s["m"][k].double().cpu().numpy() - m) <= 4e-7 * size).all(), ("m", k)
            size = v0[k] + grads[k] ** 2
            assert (np.abs(s["v"][k].double().cpu().numpy() - v) <= 4e-7 * size).all(), ("v", k)
            continue
        errors = {"m": 4e-7 * (np.abs(m0[k]) + np.abs(grads[k])), "v": 4e-7 * np.sqrt(v)}
        for name, scales, value, root in (("m", "ms", m, False), ("v", "vs", np.sqrt(v), True)):
            want, scale, unsure = ref.encode(value, t, root, errors[name])
            assert np.allclose(s[scales][k].double().cpu().numpy(), scale, rtol=2e-6, atol=0), (name, k)
            got = held([s[name][k]], [s[scales][k]])[0]
            differ = np.abs(got - want) > 1e-5 * np.abs(want)
            assert not (differ & ~unsure).any(), (name, k)
            off += int(differ.sum())
    assert off <= 0.002 * sum(len(p) for p in p0) + 2


SIZES = [1, 2, 3, 4, 5, 0, 63, 255, 256, 257, 1000, 4095, 4096, 4097, 9001]


@pytest.mark.parametrize("dtype,master", [("f32", False), ("f16", False), ("bf16", False), ("f16", True),
                                          ("bf16", True), ("f32", True)])
@pytest.mark.parametrize("bits", [32, 8])
def test_step(dtype, master, bits):
    for shift, clip, scale in ((0, None, 1.0), (1, 0.1, 0.25)):
        check(make(SIZES, dtype, bits, master, seed=shift, shift=shift), dtype, bits, clip=clip,
              grad_scale=scale, what=(dtype, master, bits, shift))


@pytest.mark.parametrize("bits", [32, 8])
def test_more_tensors_than_one_launch_holds(bits):
    check(make([7 + 3 * k for k in range(700)], "f32", bits, False), "f32", bits, clip=0.5, what=(700, bits))


def test_first_step():
    for bits in (32, 8):
        s = make([300], "f32", bits, False)
        for k in ("m", "v", "ms", "vs"):
            if s[k]:
                s[k] = [torch.zeros(t.shape, device="cuda").to(t.dtype) for t in s[k]]
        check(s, "f32", bits, t0=0, what=bits)


def test_rounding_follows_slow_moments():
    """g^2 slightly above v: each step moves v by far less than half a code, and over many steps
    the held moments still follow the exact ones, on the mean over a block, to the 12 % that a
    code's step is at most and 2 % on the mean."""
    import aware_conv_amd as A
    n = 4096
    g = torch.full((n,), 2e-3, device="cuda")
    g[::256] = 4e-3  # sets the scale of each block
    s = {"p": torch.zeros(n, device="cuda"), "m": torch.zeros(n, dtype=torch.uint8, device="cuda"),
         "v": torch.zeros(n, dtype=torch.uint8, device="cuda")}
    m, v = s["m"].view(torch.float8_e4m3fn), s["v"].view(torch.float8_e4m3fn)
    ms, vs = torch.zeros(n // 256, device="cuda"), torch.zeros(n // 256, device="cuda")
    step = torch.zeros(1, dtype=torch.int32, device="cuda")
    for _ in range(400):
        A.adamw_step([s["p"]], [g], [m], [v], step, scales=([ms], [vs]), **HYPER)
    exact = 2e-3 * np.sqrt(1 - 0.999 ** 400)
    got = held([v], [vs])[0].reshape(-1, 256)[:, 1:]
    assert abs(got.mean() / exact - 1) < 0.02 and (np.abs(got / exact - 1) < 0.3).all()
    got = held([m], [ms])[0].reshape(-1, 256)[:, 1:]
    assert abs(got.mean() / 2e-3 - 1) < 0.02


def test_values_that_are_not_finite_stay_where_they_are():
    import aware_conv_amd as A
    for bits in (32, 8):
        s = make([600], "f32", bits, False)
        s["g"][0][5], s["g"][0][300] = float("nan"), float("inf")
        step = torch.zeros(1, dtype=torch.int32, device="cuda")
        A.adamw_step(s["p"], s["g"], s["m"], s["v"], step, scales=(s["ms"], s["vs"]) if bits == 8 else None,
                     **HYPER)
        bad = torch.zeros(600, dtype=torch.bool, device="cuda")
        bad[5] = bad[300] = True
        for k in ("p", "m", "v"):
            t = s[k][0].float()
            assert torch.isfinite(t[~bad]).all(), (bits, k)
        assert s["m"][0].float()[5].isnan()
        if bits == 8:
            assert s["m"][0].float()[300].isnan() and torch.isfinite(s["ms"][0]).all()


def test_a_step_without_a_finite_norm_is_left_out():
    import aware_conv_amd as A
    for bits in (32, 8):
        s = make([600, 5], "f16", bits, True)
        s["g"][1][3] = float("inf")
        old = {k: [t.clone() for t in s[k]] for k in s if s[k]}
        step = torch.full((1,), 6, dtype=torch.int32, device="cuda")
        norm = A.adamw_grad_norm(s["g"])
        assert not torch.isfinite(norm).any()
        A.adamw_step(s["p"], s["g"], s["m"], s["v"], step, masters=s["w"], grad_norm=norm, max_norm=1.0,
                     scales=(s["ms"], s["vs"]) if bits == 8 else None, **HYPER)
        assert int(step) == 6
        for k, ts in old.items():
            for a, b in zip(s[k], ts):
                assert torch.equal(a.view(torch.uint8), b.view(torch.uint8)), k


def test_norm_of_extreme_gradients():
    import aware_conv_amd as A
    g = [torch.full((100000,), 1e30, device="cuda"), torch.full((3,), 1e-30, device="cuda")]
    want = ref.norm(arrays(g))
    assert abs(float(A.adamw_grad_norm(g)) - want) <= 2.0 ** -23 * want
    tiny = [torch.full((1000,), 1e-30, device="cuda")]
    want = ref.norm(arrays(tiny))
    assert abs(float(A.adamw_grad_norm(tiny)) - want) <= 2.0 ** -23 * want
    scale = torch.tensor([0.5], device="cuda")
    assert abs(float(A.adamw_grad_norm(tiny, grad_scale=scale)) - want / 2) <= 2.0 ** -23 * want


def test_device_scalars_and_graph():
    """Learning rate, gradient scale, norm and step number are read at replay."""
    import aware_conv_amd as A
    for bits in (32, 8):
        a, b = (make([5000, 77], "bf16", bits, True) for _ in range(2))
        step = [torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2)]
        lr = torch.tensor([1e-2], device="cuda")
        scale = torch.tensor([0.5], device="cuda")
        ws = torch.empty(4096, dtype=torch.uint8, device="cuda")
        norm = torch.empty(1, device="cuda")

        def run(s, step, lr, scale):
            n = A.adamw_grad_norm(s["g"], grad_scale=scale, norm=norm, workspace=ws)
            A.adamw_step(s["p"], s["g"], s["m"], s["v"], step, masters=s["w"], grad_norm=n, max_norm=0.3,
                         scales=(s["ms"], s["vs"]) if bits == 8 else None, grad_scale=scale, workspace=ws,
                         **dict(HYPER, lr=lr))

        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            run(a, step[0], lr, scale)
        for k in range(4):
            lr.fill_(1e-2 / (k + 1))
            scale.fill_(0.5 + k)
            ws.fill_(0x5a)
            torch.cuda.synchronize()
            graph.replay()
            torch.cuda.synchronize()
            run(b, step[1], float(np.float32(1e-2 / (k + 1))), 0.5 + k)
            assert int(step[0]) == int(step[1]) == k + 1
            for key in ("p", "w", "m", "v", "ms", "vs"):
                for x, y in zip(a[key] or [], b[key] or []):
                    assert torch.equal(x.view(torch.uint8), y.view(torch.uint8)), (bits, k, key)


def test_optimizer_against_its_formula_and_reload():
    import aware_conv_amd as A
    g = torch.Generator().manual_seed(3)
    shapes = [(7, 5), (300,), (2, 3, 4)]
    start = [torch.randn(s, generator=g) for s in shapes]
    ps = [torch.nn.Parameter(t.cuda()) for t in start]
    opt = A.AdamW(ps, max_norm=2.0, **HYPER)
    x = [t.double().numpy() for t in start]
    m, v = [np.zeros(s) for s in shapes], [np.zeros(s) for s in shapes]
    count = [0, 0, 0]
    for t in range(1, 7):
        grads = [torch.randn(s, generator=g) for s in shapes]
        if t in (3, 4):
            grads[1] = None  # this parameter stays behind
        for p, d in zip(ps, grads):
            p.grad = None if d is None else d.cuda()
        opt.step()
        live = [d.double().numpy() for d in grads if d is not None]
        c = min(1.0, 2.0 / (ref.norm(live) + 1e-6))
        for k, d in enumerate(grads):
            if d is not None:
                count[k] += 1
                x[k], m[k], v[k] = ref.adamw(x[k], d.double().numpy() * c, m[k], v[k], count[k], **HYPER)
        if t == 4:  # a new optimizer goes on from the saved states
            saved = opt.state_dict()
            opt = A.AdamW(ps, max_norm=2.0, **HYPER)
            opt.load_state_dict(saved)
    for p, want in zip(ps, x):
        assert np.abs(p.detach().double().cpu().numpy() - want).max() <= 1e-5 * np.abs(want).max()
    assert [int(opt.state[p]["step"]) for p in ps] == count


def test_optimizer_reloads_codes_and_masters():
    import aware_conv_amd as A
    g = torch.Generator().manual_seed(4)
    w = torch.randn(1000, generator=g)
    runs = []
    for reload in (False, True):
        p = torch.nn.Parameter(w.cuda().half())
        opt = A.AdamW([p], bits=8, skip_nonfinite=True, **HYPER)
        for t in range(4):
            p.grad = (torch.randn(1000, generator=torch.Generator().manual_seed(t)) * 0.1).half().cuda()
            opt.step()
            if reload and t == 1:
                saved = opt.state_dict()
                opt = A.AdamW([p], bits=8, skip_nonfinite=True, **HYPER)
                opt.load_state_dict(saved)
        st = opt.state[p]
        assert st["exp_avg"].dtype == torch.float8_e4m3fn and st["master"].dtype == torch.float32
        runs.append([p.detach().clone(), st["master"], st["exp_avg"].view(torch.uint8), st["exp_avg_sq_scale"]])
    assert all(torch.equal(a, b) for a, b in zip(*runs))
