"""The 8-bit moments of the AdamW step bit for bit.

What codes and scales are formed from is defined to the last bit
(include/adamw.h): fp32 operations in a given order, each rounded by itself.
numpy's float32 follows that order here, so nothing may differ, over any number
of steps, though a code is a discontinuous function of what it is formed from."""
import importlib.util
import os

import numpy as np
import pytest
import torch

import seq_reference as ref

pytestmark = pytest.mark.gpu

F = np.float32
DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
HYPER = {"lr": 3e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.1}
PERF = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "perf", "operators.py")


def factor(norm, max_norm, grad_scale):
    if norm is None:
        return F(grad_scale)
    return F(grad_scale) * min(F(1), F(max_norm) / (F(norm) + F(1e-6)))


def moments(g, m, ms, v, vs, k):
    """New m and sqrt(v) from the values of the codes, their scales and the gradient, all fp32."""
    n = len(g)
    b1, b2 = HYPER["betas"]
    g = g * k
    m = m * np.repeat(ms, 256)[:n]
    s = v * np.repeat(vs, 256)[:n]
    m = F(b1) * m + F(1 - b1) * g
    v = F(b2) * (s * s) + (F(1 - b2) * g) * g
    return m, np.sqrt(v)


def encode(values, t, root):
    """(values the codes stand for in units of the scale, scales)."""
    n = len(values)
    pad = np.zeros(-(-n // 256) * 256, dtype=F)
    pad[:n] = values
    blocks = pad.reshape(-1, 256)
    scales = np.abs(blocks).max(1) * F(1 / 448)
    scales[scales < F(2.0 ** -126)] = 0
    inv = np.where(scales > 0, F(1) / np.where(scales > 0, scales, F(1)), F(0)).astype(F)
    x = np.abs(blocks * inv[:, None]).ravel()[:n]
    d = ref.dither(n, t, 2 ** 31 if root else 0).astype(F)  # exact: 24 bits
    step = np.ldexp(F(1), np.frexp(np.maximum(x, F(2.0 ** -6)))[1] - 4).astype(F)
    q = np.minimum(np.floor(x / step + d) * step, F(448))
    if root:
        q = np.where((x > 0) & (q == 0), F(2.0 ** -9), q)
    return np.copysign(q, values), scales


def make(sizes, dtype, seed, shift):
    g = torch.Generator().manual_seed(seed)

    def place(t):
        flat = torch.zeros(t.numel() + shift, dtype=t.dtype, device="cuda")
        flat[shift:] = t.cuda()
        return flat[shift:]

    s = {k: [] for k in ("p", "g", "m", "v", "w", "ms", "vs")}
    for n in sizes:
        w = torch.randn(n, generator=g) * 0.1
        s["w"].append(place(w))
        s["p"].append(place(w.to(DT[dtype])))
        s["g"].append(place((torch.randn(n, generator=g) * 1e-2).to(DT[dtype])))
        codes = torch.randint(0, 127, (2, n), generator=g, dtype=torch.uint8)
        codes[0] |= (torch.rand(n, generator=g) < 0.5).to(torch.uint8) * 128
        s["m"].append(place(codes[0]).view(torch.float8_e4m3fn))
        s["v"].append(place(codes[1]).view(torch.float8_e4m3fn))
        for k in ("ms", "vs"):
            s[k].append(place(torch.rand(-(-n // 256), generator=g) * 1e-4))
    return s


def values(ts):
    return [t.float().cpu().numpy() for t in ts]


@pytest.mark.parametrize("dtype", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("master", [False, True])
@pytest.mark.parametrize("max_norm,grad_scale", [(None, 1.0), (None, 0.3), (1.0, 1.0), (0.7, 0.25)])
def test_codes_and_scales_are_those_of_the_definition(dtype, master, max_norm, grad_scale):
    import aware_conv_amd as A
    what = (dtype, master, max_norm, grad_scale)
    print("\ncase codes %s" % (what,), flush=True)
    s = make([1, 255, 256, 257, 4095, 4097, 30011, 200003], dtype, 5, shift=1 if grad_scale == 0.25 else 0)
    step = torch.full((1,), 4, dtype=torch.int32, device="cuda")
    for t in (5, 6, 7):
        g, m0, v0, ms, vs = (values(s[k]) for k in ("g", "m", "v", "ms", "vs"))
        p0 = [a.astype(np.float64) for a in values(s["w"] if master else s["p"])]
        norm = None
        if max_norm is not None:
            norm = A.adamw_grad_norm(s["g"], grad_scale=grad_scale)
        A.adamw_step(s["p"], s["g"], s["m"], s["v"], step, masters=s["w"] if master else None,
                     scales=(s["ms"], s["vs"]), grad_scale=grad_scale, grad_norm=norm, max_norm=max_norm, **HYPER)
        torch.cuda.synchronize()
        k = factor(None if norm is None else float(norm), max_norm, grad_scale)
        exact = grad_scale * (1.0 if norm is None else min(1.0, max_norm / (float(norm) + 1e-6)))
        for j in range(len(g)):
            m, r = moments(g[j], m0[j], ms[j], v0[j], vs[j], k)
            for name, scale, value, root in (("m", "ms", m, False), ("v", "vs", r, True)):
                q, size = encode(value, t, root)
                assert np.array_equal(s[scale][j].cpu().numpy(), size), (t, name, j)
                assert np.array_equal(s[name][j].float().cpu().numpy(), q), (t, name, j)
            # the parameter to the tolerance of tests/test_gpu_adamw.py, from the moments as held before
            held = [a[j].astype(np.float64) * np.repeat(b[j].astype(np.float64), 256)[:len(g[j])]
                    for a, b in ((m0, ms), (v0, vs))]
            p, _, _ = ref.adamw(p0[j], g[j].astype(np.float64) * exact, held[0], held[1] ** 2, t, **HYPER)
            got = (s["w"] if master else s["p"])[j].double().cpu().numpy()
            bound = 2e-7 * np.abs(p0[j]) + 2e-6 * np.abs(p - p0[j] * (1 - HYPER["lr"] * HYPER["weight_decay"]))
            if not master:
                half = {"f32": 2.0 ** -24, "f16": 2.0 ** -11, "bf16": 2.0 ** -8}[dtype]
                bound = bound + half * np.abs(p) + (2.0 ** -25 if dtype == "f16" else 0)
            assert (np.abs(got - p) <= bound).all(), (t, "p", j)


def test_the_largest_of_a_block():
    """Steps whose dither is below 2^-20 at one element of a block: its largest magnitude there is
    held as the definition says, 448 where its quotient is, else the code below."""
    import aware_conv_amd as A
    g = torch.Generator().manual_seed(6)
    for t, at, moment in ((12653, 85, "m"), (13524, 13, "m"), (6079, 255, "v"), (45404, 13, "v")):
        assert ref.dither(256, t, 0 if moment == "m" else 2 ** 31)[at] < 2.0 ** -20
        n = 256 * 64
        grad = torch.rand(n, generator=g) * 1e-3 + 1e-3
        grad[at::256] *= 3  # the largest of each block
        grad = grad.cuda()
        m, v = (torch.zeros(n, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn) for _ in range(2))
        ms, vs = torch.zeros(64, device="cuda"), torch.zeros(64, device="cuda")
        p = torch.zeros(n, device="cuda")
        step = torch.full((1,), t - 1, dtype=torch.int32, device="cuda")
        # element k of every block but the first has another dither: one tensor per block
        A.adamw_step(list(p.split(256)), list(grad.split(256)), list(m.split(256)), list(v.split(256)), step,
                     scales=(list(ms.split(1)), list(vs.split(1))), **HYPER)
        zero = np.zeros(256, dtype=F)
        seen = set()
        for b in range(64):
            a, r = moments(grad[256 * b:256 * b + 256].cpu().numpy(), zero, zero[:1], zero, zero[:1], F(1))
            for name, codes, scales, value in (("m", m, ms, a), ("v", v, vs, r)):
                q, size = encode(value, t, name == "v")
                assert np.array_equal(codes[256 * b:256 * b + 256].float().cpu().numpy(), q), (t, name, b)
                assert float(scales[b]) == float(size[0])
                if name == moment:
                    seen.add(float(q[at]))
        assert 448.0 in seen and seen <= {448.0, 416.0}


@pytest.mark.parametrize("dtype,master", [("f32", False), ("bf16", True), ("f16", False)])
def test_two_steps_agree_with_the_plain_form(dtype, master):
    """The torch form of perf/operators.py, where the gradients are not clipped (its norm is an fp32
    sum): the same codes and scales after two steps in place."""
    spec = importlib.util.spec_from_file_location("perf_operators", PERF)
    ops = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(ops)
    case = {"kind": "adamw", "tensors": 23, "smallest": 1, "largest": 200003, "dtype": dtype, "bits": 8,
            "clip": False, "master": master}
    out = []
    for ops.own in (False, True):
        s = ops.prepare(case, 3)
        ops.run(s)
        out.append(ops.run(s))
    torch.cuda.synchronize()
    for k in ("m", "v", "ms", "vs"):
        assert torch.equal(out[0][k].float(), out[1][k].float()), k
    # two fp32 evaluations of one formula: 2e-6 of the largest update's terms, |p| < 0.12
    top = out[0]["w" if master else "p"].float()
    near = (top - out[1]["w" if master else "p"].float()).abs()
    half = 0 if master or dtype == "f32" else 2.0 ** -11
    assert (near <= 1e-6 + 2 * half * top.abs()).all()


def test_tensors_that_only_an_iterator_makes():
    """Gradients converted on the way into the call, against the same in a list."""
    import aware_conv_amd as A
    out = []
    for make_list in (True, False):
        g = torch.Generator(device="cuda").manual_seed(1)
        p = [torch.randn(5000 + k, generator=g, device="cuda") for k in range(20)]
        half = [torch.randn(5000 + k, generator=g, device="cuda").half() for k in range(20)]
        m, v = ([torch.zeros_like(t) for t in p] for _ in range(2))
        grads = (t.float() for t in half)
        step = torch.zeros(1, dtype=torch.int32, device="cuda")
        A.adamw_step(p, list(grads) if make_list else grads, m, v, step, **HYPER)
        out.append(p + m + v)
    assert all(torch.equal(a, b) for a, b in zip(*out))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_copied_optimizer_goes_on_as_the_first(bits):
    import copy
    import aware_conv_amd as A
    p = [torch.nn.Parameter(torch.randn(n, generator=torch.Generator().manual_seed(n)).half().cuda())
         for n in (300, 5)]
    opt = A.AdamW(p, bits=bits, max_norm=0.1, grad_scale=0.5, **HYPER)

    def steps(p, opt, seed):
        for t in range(2):
            for k, w in enumerate(p):
                g = torch.Generator().manual_seed(100 * seed + 10 * t + k)
                w.grad = torch.randn(w.shape, generator=g).half().cuda()
            opt.step()

    steps(p, opt, 1)
    p2, opt2 = copy.deepcopy((p, opt))
    steps(p, opt, 2)
    steps(p2, opt2, 2)
    for a, b in zip(p, p2):
        assert torch.equal(a, b)
        for n, t in opt.state[a].items():
            assert torch.equal(t.view(torch.uint8), opt2.state[b][n].view(torch.uint8)), n
    assert opt2.state[p2[0]]["step"] is opt2.state[p2[1]]["step"]
