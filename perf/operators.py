"""Cases of the sequence and training operators, for measuring them.

Two operators, each with its companions:

* the gated linear recurrence (``gscan_fwd``, ``gscan_bwd``, ``gscan_step``)

      L = -c softplus(lam) sig(r),  a = exp(L),  w = sqrt(1 - a^2)
      h_t = a_t h_{t-1} + w_t sig(i_t) x_t

  over planes ("bct": time contiguous, NCHW planes flattened in raster order)
  or tokens ("btc": channels contiguous), and one token at a time on a cache
  of states;

* the AdamW step over many tensors (``adamw_step``) with states in 32 bits or
  in 8 (e4m3 codes of m and sqrt(v) with one scale per 256 elements), and the
  global gradient norm that clips it (``adamw_grad_norm``).

``own`` selects the framework's kernels; otherwise ``run`` computes the same
in elementary torch operations in fp32.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
DECAY = 8.0           # c in L = -c softplus(lam) sig(r)
BLOCK = 256           # elements per scale of the 8-bit states
HYPER = {"lr": 1e-3, "betas": (0.9, 0.999), "eps": 1e-8, "weight_decay": 0.05}
MAX_NORM = 1.0
# dither of the 8-bit rounding: golden-ratio steps over the elements, plastic-
# number steps over the training steps, in 32-bit fixed point
PHI_INDEX, PHI_STEP, PHI_V = 2654435769, 3242174889, 1 << 31


def listed():
    return [
        # one decoded token of one sequence: launch latency alone
        {"name": "token_1x384_f32", "kind": "step", "B": 1, "C": 384, "dtype": "f32"},
        # a full serving batch's next token
        {"name": "token_512x4096_bf16", "kind": "step", "B": 512, "C": 4096, "dtype": "bf16"},
        # the small planes of the stage-3 workload: short rows, many of them
        {"name": "planes_stage3_f32", "kind": "scan", "layout": "bct", "B": 64, "C": 384, "T": 14 * 14,
         "dtype": "f32", "train": True, "packed": True, "reverse": False, "state": False, "ragged": False},
        # the fp16 stage-1 workload's planes, scanned from the end (the second direction of a
        # two-way mixer)
        {"name": "planes_stage1_f16", "kind": "scan", "layout": "bct", "B": 128, "C": 96, "T": 56 * 56,
         "dtype": "f16", "train": True, "packed": True, "reverse": True, "state": False, "ragged": False},
        # the high-resolution workload: 512 rows of 262144
        {"name": "planes_highres_f32", "kind": "scan", "layout": "bct", "B": 8, "C": 64, "T": 512 * 512,
         "dtype": "f32", "train": True, "packed": False, "reverse": False, "state": False, "ragged": False},
        # a training step over token sequences
        {"name": "tokens_8x4096_bf16", "kind": "scan", "layout": "btc", "B": 8, "C": 2048, "T": 4096,
         "dtype": "bf16", "train": True, "packed": True, "reverse": False, "state": False, "ragged": False},
        # one long prompt read into a state, odd length
        {"name": "prompt_1x65521_bf16", "kind": "scan", "layout": "btc", "B": 1, "C": 2560, "T": 65521,
         "dtype": "bf16", "train": False, "packed": True, "reverse": False, "state": True, "ragged": False},
        # padded sequences of many lengths (one empty), odd channels, continued from states
        {"name": "ragged_24x1000_f16", "kind": "scan", "layout": "btc", "B": 24, "C": 999, "T": 1000,
         "dtype": "f16", "train": True, "packed": False, "reverse": False, "state": True, "ragged": True},
        # the parameters of eighteen such layers: ninety small tensors, clipped
        {"name": "adamw_layers_f32", "kind": "adamw", "tensors": 90, "smallest": 96, "largest": 76800,
         "dtype": "f32", "bits": 32, "clip": True, "master": False},
        # a model's large matrices in fp32
        {"name": "adamw_large_f32", "kind": "adamw", "tensors": 16, "smallest": 1 << 20, "largest": 1 << 24,
         "dtype": "f32", "bits": 32, "clip": False, "master": False},
        # odd sizes, 8-bit states, clipped
        {"name": "adamw_odd_f32_8bit", "kind": "adamw", "tensors": 37, "smallest": 1, "largest": 1000003,
         "dtype": "f32", "bits": 8, "clip": True, "master": False},
        # mixed precision: bf16 parameters and gradients, fp32 masters, 8-bit states
        {"name": "adamw_large_bf16_8bit", "kind": "adamw", "tensors": 24, "smallest": 1 << 20, "largest": 1 << 24,
         "dtype": "bf16", "bits": 8, "clip": True, "master": True},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["step", "scan", "scan", "scan", "adamw", "adamw"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind == "step":
        return {"kind": kind, "B": _log(rng, 1, 512), "C": _log(rng, 64, 4097), "dtype": dtype}
    if kind == "adamw":
        lo = _log(rng, 1, 100000)
        return {"kind": kind, "tensors": _log(rng, 2, 150), "smallest": lo,
                "largest": _log(rng, max(lo, 1000), 1 << 20), "dtype": dtype, "bits": rng.choice([8, 32]),
                "clip": rng.random() < 0.5, "master": dtype != "f32" and rng.random() < 0.7}
    layout = rng.choice(["bct", "btc"])
    T = _log(rng, 2, 200000)
    C = _log(rng, 16, 4100)
    while C * T > 1 << 25:
        C = max(16, C // 2 + rng.randrange(2))
    B = max(1, min(_log(rng, 1, 64), (1 << 26) // (C * T)))
    return {"kind": kind, "layout": layout, "B": B, "C": C, "T": T, "dtype": dtype,
            "train": rng.random() < 0.6, "packed": rng.random() < 0.5, "reverse": rng.random() < 0.3,
            "state": rng.random() < 0.5, "ragged": rng.random() < 0.4}


def _sizes(case):
    """Elements of each tensor, spread evenly over the logarithm between the two ends."""
    n, lo, hi = case["tensors"], case["smallest"], case["largest"]
    return [int(round(lo * (hi / lo) ** (k / max(1, n - 1)))) for k in range(n)]


def _lam(C, g, dev):
    # decay at a fully open gate uniform in 0.9..0.999
    a = 0.9 + 0.099 * torch.rand(C, generator=g, device=dev)
    s = -torch.log(a) / DECAY
    return torch.log(torch.expm1(s))


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    td = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = dict(case)
    if case["kind"] == "step":
        B, C = case["B"], case["C"]
        proj = randn(B, 3 * C, dtype=td)
        s["x"], s["r"], s["i"] = proj.chunk(3, dim=1)
        s["lam"] = _lam(C, g, dev)
        slots = B + B // 4 + 1
        s["cache"] = randn(slots, C)
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:B].to(torch.int32)
        return s
    if case["kind"] == "scan":
        B, C, T = case["B"], case["C"], case["T"]
        shape = (B, C, T) if case["layout"] == "bct" else (B, T, C)
        if case["packed"]:  # x and both gates come from one projection
            dim = 1 if case["layout"] == "bct" else 2
            wide = list(shape)
            wide[dim] = 3 * C
            s["proj"] = randn(*wide, dtype=td)
            s["x"], s["r"], s["i"] = s["proj"].chunk(3, dim=dim)
            s["dim"] = dim
        else:
            s["proj"] = None
            s["x"], s["r"], s["i"] = (randn(*shape, dtype=td) for _ in range(3))
        s["lam"] = _lam(C, g, dev)
        s["h0"] = randn(B, C) if case["state"] else None
        s["lengths"] = None
        if case["ragged"]:
            n = torch.randint(1, T + 1, (B,), generator=g, device=dev)
            n[0] = T
            n[B // 2:B // 2 + 1] = 0 if B > 1 else T
            s["lengths"] = n.to(torch.int32)
        if case["train"]:
            s["dh"] = randn(*shape, dtype=td)
            s["dh_last"] = randn(B, C) if case["state"] else None
        return s
    sizes = _sizes(case)
    pads = [-(-n // BLOCK) * BLOCK for n in sizes]  # every tensor starts on a block of the flat buffers
    starts = [sum(pads[:k]) for k in range(len(pads))]
    total = sum(pads)
    inside = torch.zeros(total, dtype=torch.bool, device=dev)
    at = torch.zeros(total, dtype=torch.int32, device=dev)
    for o, n in zip(starts, sizes):
        inside[o:o + n] = True
        at[o:o + n] = torch.arange(n, dtype=torch.int32, device=dev)
    s["at"] = at

    def flat(scale):
        return randn(total) * scale * inside

    master = flat(0.02)
    s["g"] = flat(1e-3).to(td)
    m, v = flat(1e-3), (flat(1e-3).square() + 1e-8) * inside
    s["p"] = master.to(td)
    s["w"] = master if case["master"] else None
    s["ms"] = s["vs"] = None
    if case["bits"] == 8:
        at_step = torch.full((1,), 9, dtype=torch.int32, device=dev)
        m, s["ms"] = _encode(m, at, at_step, 0)
        v, s["vs"] = _encode(v.sqrt(), at, at_step, PHI_V)
    s["m"], s["v"] = m, v
    s["step"] = torch.full((1,), 9, dtype=torch.int32, device=dev)

    def views(t, per=1):
        return None if t is None else [t[o // per:o // per + -(-n // per)] for o, n in zip(starts, sizes)]

    s["lists"] = {k: views(s[k]) for k in ("p", "g", "m", "v", "w")}
    s["lists"]["ms"], s["lists"]["vs"] = views(s["ms"], BLOCK), views(s["vs"], BLOCK)
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _scan(a, b):
    """Inclusive scan of h_t = a_t h_{t-1} + b_t over the last axis, by doubling."""
    T, reach = a.shape[-1], 1
    a, b = a.clone(), b.clone()
    while reach < T:  # log2(T) passes: a recurrence has no elementwise form
        b = torch.cat([b[..., :reach], b[..., reach:] + a[..., reach:] * b[..., :-reach]], -1)
        a = torch.cat([a[..., :reach], a[..., reach:] * a[..., :-reach]], -1)
        reach *= 2
    return b


def _ordered(s, t):
    """[B, C, T] in fp32, time in scan order (padding behind the valid part)."""
    t = t.float() if s["layout"] == "bct" else t.float().transpose(1, 2)
    if s["reverse"]:
        t = t.flip(-1) if s["lengths"] is None else torch.gather(t, 2, _turned(s).expand_as(t))
    return t.contiguous()


def _turned(s):
    """Positions that reverse the valid part of each sequence and keep the rest."""
    n = s["lengths"].long().view(-1, 1, 1)
    t = torch.arange(s["T"], device=n.device).view(1, 1, -1)
    return torch.where(t < n, n - 1 - t, t)


def _stored(s, t):
    """Back from scan order, in the layout and type of the tensors."""
    if s["reverse"]:
        t = t.flip(-1) if s["lengths"] is None else torch.gather(t, 2, _turned(s).expand_as(t))
    t = t if s["layout"] == "bct" else t.transpose(1, 2)
    return t.to(DTYPES[s["dtype"]]).contiguous()


def _plain_scan(s):
    x, r, i = (_ordered(s, s[k]) for k in ("x", "r", "i"))
    B, C, T = x.shape
    soft = torch.nn.functional.softplus(s["lam"]).view(1, C, 1)
    sr, si = torch.sigmoid(r), torch.sigmoid(i)
    L = -DECAY * soft * sr
    w = torch.sqrt(-torch.expm1(2 * L))
    a = torch.exp(L)
    b = w * si * x
    live = None
    if s["lengths"] is not None:
        live = torch.arange(T, device=x.device).view(1, 1, T) < s["lengths"].view(B, 1, 1)
        a, b = torch.where(live, a, 1.0), torch.where(live, b, 0.0)
    h0 = s["h0"] if s["h0"] is not None else torch.zeros(B, C, device=x.device)
    first = b[..., :1] + a[..., :1] * h0.unsqueeze(-1)
    h = _scan(a, torch.cat([first, b[..., 1:]], -1))
    out = {"h": _stored(s, h if live is None else torch.where(live, h, 0.0)), "h_last": h[..., -1].contiguous()}
    if not s["train"]:
        return out
    dh = _ordered(s, s["dh"])
    if live is not None:
        dh = torch.where(live, dh, 0.0)
    if s["dh_last"] is not None:
        dh = torch.cat([dh[..., :-1], dh[..., -1:] + s["dh_last"].unsqueeze(-1)], -1)
    after = torch.cat([a[..., 1:], torch.ones_like(a[..., :1])], -1)
    gr = _scan(after.flip(-1), dh.flip(-1)).flip(-1)
    before = torch.cat([h0.unsqueeze(-1), h[..., :-1]], -1)
    dL = gr * (a * before - torch.where(w > 0, si * x * a * a / w, 0.0))
    parts = {"dx": gr * w * si, "dr": dL * L * torch.sigmoid(-r), "di": gr * w * x * si * torch.sigmoid(-i)}
    dlam = dL * (-DECAY) * sr * torch.sigmoid(s["lam"]).view(1, C, 1)
    if live is not None:
        parts = {k: torch.where(live, t, 0.0) for k, t in parts.items()}
        dlam = torch.where(live, dlam, 0.0)
    out.update({k: _stored(s, t) for k, t in parts.items()})
    out["dlam"] = dlam.sum((0, 2))
    out["dh0"] = a[..., 0] * gr[..., 0]
    return out


def _plain_step(s):
    x, r, i = (s[k].float() for k in ("x", "r", "i"))
    L = -DECAY * torch.nn.functional.softplus(s["lam"]) * torch.sigmoid(r)
    at = s["slots"].long()
    h = torch.exp(L) * s["cache"][at] + torch.sqrt(-torch.expm1(2 * L)) * torch.sigmoid(i) * x
    s["cache"][at] = h
    return {"h": h.to(DTYPES[s["dtype"]]), "cache": s["cache"]}


def _encode(t, at, step, turn):
    """Codes (e4m3) and scales of `t`, one scale per block, rounded up or down by the dither.
    A value that is not zero keeps a code that is not zero where turn is PHI_V (sqrt(v))."""
    scale = t.view(-1, BLOCK).abs().amax(1) / 448.0
    x = (t.view(-1, BLOCK) * torch.where(scale > 0, 1.0 / scale, 0.0).unsqueeze(1)).view(-1)
    u = (at.long() * PHI_INDEX + step.long() * PHI_STEP + turn) & 0xFFFFFFFF
    d = (u >> 8).to(t.dtype) * 2.0 ** -24
    y = x.abs()
    ulp = torch.exp2(torch.floor(torch.log2(y.clamp_min(2.0 ** -6))) - 3)
    # log2 may round up across a power of two
    ulp = torch.where(ulp * 8 > y.clamp_min(2.0 ** -6), ulp / 2, ulp)
    q = (torch.floor(y / ulp + d) * ulp).clamp_max(448.0)
    if turn:
        q = torch.where((x > 0) & (q == 0), 2.0 ** -9, q)
    return (q * torch.sign(x)).to(torch.float8_e4m3fn), scale


def _decode(code, scale):
    return (code.float().view(-1, BLOCK) * scale.unsqueeze(1)).view(-1)


def _plain_adamw(s):
    lr, (b1, b2), eps, decay = HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"]
    g = s["g"].float()
    out = {}
    if s["clip"]:
        out["norm"] = norm = g.square().sum().sqrt().view(1)
        g = g * (MAX_NORM / (norm + 1e-6)).clamp_max(1.0)
    s["step"] += 1
    t = s["step"].float()
    p = s["w"] if s["w"] is not None else s["p"].float()
    bits8 = s["bits"] == 8
    m = _decode(s["m"], s["ms"]) if bits8 else s["m"]
    v = _decode(s["v"], s["vs"]).square() if bits8 else s["v"]
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    c1 = -torch.expm1(t * math.log(b1))
    c2 = -torch.expm1(t * math.log(b2))
    p = p * (1 - lr * decay) - lr * (m / c1) / ((v / c2).sqrt() + eps)
    s["p"].copy_(p)
    if s["w"] is not None:
        s["w"].copy_(p)
    if bits8:
        for_m, s["ms"][:] = _encode(m, s["at"], s["step"], 0)
        for_v, s["vs"][:] = _encode(v.sqrt(), s["at"], s["step"], PHI_V)
        s["m"].copy_(for_m)
        s["v"].copy_(for_v)
    else:
        s["m"].copy_(m)
        s["v"].copy_(v)
    return dict(out, **_trained(s))


def _trained(s):
    return {k: s[k] for k in ("p", "m", "v", "w", "ms", "vs", "step") if s[k] is not None}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(state):
    s = state
    if not own:
        return {"step": _plain_step, "scan": _plain_scan, "adamw": _plain_adamw}[s["kind"]](s)
    import aware_conv_amd as A
    if s["kind"] == "step":
        h = A.gscan_step(s["x"], s["r"], s["i"], s["lam"], s["cache"], slots=s["slots"], decay=DECAY)
        return {"h": h, "cache": s["cache"]}
    if s["kind"] == "scan":
        form = {"lengths": s["lengths"], "layout": s["layout"], "reverse": s["reverse"], "decay": DECAY}
        h, h_last, states = A.gscan_fwd(s["x"], s["r"], s["i"], s["lam"], h0=s["h0"],
                                        save_states=s["train"], **form)
        out = {"h": h, "h_last": h_last}
        if s["train"]:
            grads = None
            if s["proj"] is not None:  # the gradient of the projection, written in place of its parts
                dproj = torch.empty_like(s["proj"])
                grads = dict(zip(("dx", "dr", "di"), dproj.chunk(3, dim=s["dim"])))
            out.update(A.gscan_bwd(s["x"], s["r"], s["i"], s["lam"], states, s["dh"], dh_last=s["dh_last"],
                                   grads=grads, **form))
        return out
    k = s["lists"]
    norm = A.adamw_grad_norm(k["g"]) if s["clip"] else None
    A.adamw_step(k["p"], k["g"], k["m"], k["v"], s["step"], masters=k["w"],
                 scales=(k["ms"], k["vs"]) if s["bits"] == 8 else None,
                 grad_norm=norm, max_norm=MAX_NORM if s["clip"] else None, **HYPER)
    return dict({} if norm is None else {"norm": norm}, **_trained(s))


def work(case):
    e = SIZES[case["dtype"]]
    if case["kind"] == "step":
        n = case["B"] * case["C"]
        return {"bytes": n * (4 * e + 8) + 4 * case["C"] + 4 * case["B"], "flops": 30 * n}
    if case["kind"] == "scan":
        rows = case["B"] * case["C"]
        n = rows * case["T"]
        small = 4 * case["C"] + rows * 4 * (1 + case["state"])
        if not case["train"]:
            return {"bytes": 4 * n * e + small, "flops": 30 * n}
        return {"bytes": 8 * n * e + small + 4 * case["C"] + rows * 4 * (1 + case["state"]), "flops": 90 * n}
    n = sum(_sizes(case))
    state = 16 if case["bits"] == 32 else 4 + 16 / BLOCK
    weights = (8 + e) if case["master"] else 2 * e
    return {"bytes": n * (weights + e + state), "flops": 20 * n}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits
# ---------------------------------------------------------------------------

def _exact_recurrence(a, b, first):
    """h_t = a_t h_{t-1} + b_t with h_{-1} = first over the last axis: sequences are cut into pieces
    that advance together, then each piece is given the state it starts from."""
    T = a.shape[-1]
    piece = max(1, int(math.sqrt(T)))
    count = -(-T // piece)
    fill = count * piece - T
    a = torch.nn.functional.pad(a, (0, fill), value=1.0).unflatten(-1, (count, piece))
    b = torch.nn.functional.pad(b, (0, fill)).unflatten(-1, (count, piece))
    local, grown = torch.empty_like(b), torch.empty_like(a)
    h, p = torch.zeros_like(b[..., 0]), torch.ones_like(a[..., 0])
    for t in range(piece):
        h = a[..., t] * h + b[..., t]
        p = p * a[..., t]
        local[..., t], grown[..., t] = h, p
    start = first
    for k in range(count):
        local[..., k, :] += grown[..., k, :] * start.unsqueeze(-1)
        start = local[..., k, -1]
    return local.flatten(-2)[..., :T]


def _exact_scan(s):
    B, C, T = s["B"], s["C"], s["T"]

    def scan_order(t):
        t = t.double()
        t = t.permute(0, 2, 1) if s["layout"] == "btc" else t
        if s["reverse"]:
            t = torch.stack([torch.cat([t[b, :, :n].flip(-1), t[b, :, n:]], -1) for b, n in enumerate(lengths)])
        return t.contiguous()

    def from_order(t):
        if s["reverse"]:
            t = torch.stack([torch.cat([t[b, :, :n].flip(-1), t[b, :, n:]], -1) for b, n in enumerate(lengths)])
        return t.permute(0, 2, 1) if s["layout"] == "btc" else t

    lengths = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    alive = torch.zeros(B, 1, T, dtype=torch.bool, device=s["lam"].device)
    for b, n in enumerate(lengths):
        alive[b, :, :n] = True
    x = scan_order(s["x"])
    lam = s["lam"].double()
    rate = (DECAY * torch.log1p(torch.exp(lam)))[None, :, None]
    open_r = 1 / (1 + torch.exp(-scan_order(s["r"])))
    open_i = 1 / (1 + torch.exp(-scan_order(s["i"])))
    a = torch.exp(-rate * open_r)
    w = (-torch.expm1(-2 * rate * open_r)).sqrt()
    start = torch.zeros(B, C, dtype=torch.float64, device=x.device) if s["h0"] is None else s["h0"].double()
    held = a.masked_fill(~alive, 1.0)
    h = _exact_recurrence(held, (w * open_i * x).masked_fill(~alive, 0.0), start)
    out = {"h": from_order(h * alive), "h_last": h[..., -1].clone()}
    if not s["train"]:
        return out
    end = torch.zeros_like(start) if s["dh_last"] is None else s["dh_last"].double()
    dh = scan_order(s["dh"]).masked_fill(~alive, 0.0)
    # gradient of what enters position t: u_t = a_t (dh_t + u_{t+1}), u_T = dh_last
    u = _exact_recurrence(held.flip(-1), (held * dh).flip(-1), end).flip(-1)
    grad = dh + torch.cat([u[..., 1:], end.unsqueeze(-1)], -1)
    past = torch.cat([start.unsqueeze(-1), h[..., :-1]], -1)
    d_a = grad * past - grad * open_i * x * a / w
    d_open = d_a * a * -rate
    out["dx"] = from_order(grad * w * open_i * alive)
    out["dr"] = from_order(d_open * open_r * (1 - open_r) * alive)
    out["di"] = from_order(grad * w * x * open_i * (1 - open_i) * alive)
    d_rate = (d_a * a * -open_r * alive).sum((0, 2))
    out["dlam"] = d_rate * DECAY / (1 + torch.exp(-lam))
    out["dh0"] = u[..., 0].clone()
    return out


def _exact_code(t, at, step, turn):
    size = t.view(-1, BLOCK).abs().max(1).values / 448
    x = torch.where(size[:, None] > 0, t.view(-1, BLOCK) / size[:, None], 0).view(-1)
    d = torch.remainder(torch.remainder(at.long() * PHI_INDEX, 2 ** 32) + step * PHI_STEP + turn, 2 ** 32)
    d = torch.div(d, 256, rounding_mode="floor").double() / 2 ** 24
    fine = torch.ldexp(torch.ones_like(x), (torch.frexp(x.abs()).exponent - 1).clamp(min=-6) - 3)
    q = torch.floor(x.abs() / fine + d).mul(fine).clamp(max=448)
    if turn:
        q = torch.where((x != 0) & (q == 0), torch.full_like(q, 2.0 ** -9), q)
    return torch.copysign(q, x), size


def _exact_adamw(s):
    lr, (b1, b2), eps, decay = HYPER["lr"], HYPER["betas"], HYPER["eps"], HYPER["weight_decay"]
    t = int(s["step"]) + 1
    g = s["g"].double()
    out = {}
    if s["clip"]:
        norm = torch.linalg.vector_norm(g)
        out["norm"] = norm.view(1)
        g = g * min(1.0, MAX_NORM / (float(norm) + 1e-6))
    m, v = s["m"].double(), s["v"].double()
    if s["bits"] == 8:
        m = m * s["ms"].double().repeat_interleave(BLOCK)
        v = (v * s["vs"].double().repeat_interleave(BLOCK)) ** 2
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g ** 2
    p = (s["p"] if s["w"] is None else s["w"]).double()
    p = p - lr * decay * p - lr * (m / (1 - b1 ** t)) / (torch.sqrt(v / (1 - b2 ** t)) + eps)
    out["p"] = p
    if s["w"] is not None:
        out["w"] = p
    if s["bits"] == 8:
        m, out["ms"] = _exact_code(m, s["at"], t, 0)
        v, out["vs"] = _exact_code(v.sqrt(), s["at"], t, PHI_V)
    out["m"], out["v"], out["step"] = m, v, None
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "scan":
        return _exact_scan(s)
    if s["kind"] == "adamw":
        return _exact_adamw(s)
    x, r, i, lam = (s[k].double() for k in ("x", "r", "i", "lam"))
    a = torch.exp(-DECAY * torch.log1p(torch.exp(lam)) / (1 + torch.exp(-r)))
    at = s["slots"].long()
    h = a * s["cache"].double()[at] + (1 - a * a).sqrt() * x / (1 + torch.exp(-i))
    cache = s["cache"].double()
    cache[at] = h
    return {"h": h, "cache": cache}
