"""Cases of the state-space block's operators, for measuring them.

Three operators, which follow each other in a block over token sequences
[B, T, C]:

* the root-mean-square norm with the residual's addition (``rmsnorm_fwd``,
  ``rmsnorm_bwd``)

      s = x + residual,  y = s w / sqrt(mean(s^2) + eps)

  optionally in 8 bits: e4m3 codes and one scale per row;

* the short causal convolution (``cconv_fwd``, ``cconv_bwd``, ``cconv_step``)

      v_t = bias + sum_k w[k] x[t - K + 1 + k],  y = silu(v)

* the selective state space scan (``sscan_fwd``, ``sscan_bwd``, ``sscan_step``)

      delta = softplus(dt + dt_bias),  A = -exp(a_log)
      h_t = exp(delta A) h_{t-1} + delta x_t b_t
      y_t = (c_t . h_t + d x_t) silu(z_t)

  with N states per channel; b and c are shared by the channels of a group.

``own`` selects the framework's kernels; otherwise ``run`` computes the same
in elementary torch operations in fp32.
"""
import math

import torch

own = False

DTYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SIZES = {"f32": 4, "f16": 2, "bf16": 2}
EPS = 1e-5
TOP = 448.0  # the largest e4m3 value


def _scan_case(name, B, T, D, N, dtype, **more):
    case = {"name": name, "kind": "scan", "B": B, "T": T, "D": D, "N": N, "G": 1, "dtype": dtype,
            "train": True, "gate": True, "skip": True, "bias": True, "state": False, "ragged": False}
    case.update(more)
    return case


def listed():
    return [
        # one decoded token of one sequence through the convolution: launch latency alone
        {"name": "conv_token_1x384_f32", "kind": "conv_step", "B": 1, "C": 384, "K": 4, "dtype": "f32"},
        # a training step over token sequences; x is half of a projection
        {"name": "conv_8x4096x2048_bf16", "kind": "conv", "B": 8, "T": 4096, "C": 2048, "K": 4, "dtype": "bf16",
         "train": True, "packed": True, "state": False, "ragged": False},
        # padded sequences of many lengths (one empty), odd channels, continued from earlier inputs
        {"name": "conv_ragged_24x1000x999_f16", "kind": "conv", "B": 24, "T": 1000, "C": 999, "K": 3,
         "dtype": "f16", "train": True, "packed": False, "state": True, "ragged": True},
        # one decoded token of one sequence through the scan
        {"name": "scan_token_1x384_f32", "kind": "scan_step", "B": 1, "D": 384, "N": 16, "G": 1, "dtype": "f32"},
        # a full serving batch's next token
        {"name": "scan_token_512x4096_bf16", "kind": "scan_step", "B": 512, "D": 4096, "N": 16, "G": 1,
         "dtype": "bf16"},
        # a training step over token sequences
        _scan_case("scan_8x4096x2048_bf16", 8, 4096, 2048, 16, "bf16"),
        # one long prompt read into a state, odd length
        _scan_case("scan_prompt_1x65521x2560_bf16", 1, 65521, 2560, 16, "bf16", train=False, state=True),
        # padded sequences of many lengths (one empty), odd channels in groups, an odd number of states
        _scan_case("scan_ragged_24x1000x999_f16", 24, 1000, 999, 21, "f16", G=3, state=True, ragged=True),
        # the norm before a decoded token's projection
        {"name": "norm_token_1x384_f32", "kind": "norm", "B": 1, "T": 1, "C": 384, "dtype": "f32",
         "residual": "f32", "train": False, "bits8": False},
        # a training step's norm, the residual stream kept in fp32
        {"name": "norm_8x4096x2048_bf16", "kind": "norm", "B": 8, "T": 4096, "C": 2048, "dtype": "bf16",
         "residual": "f32", "train": True, "bits8": False},
        # a prompt on its way into a projection in 8 bits
        {"name": "norm_8bit_1x16384x4096_bf16", "kind": "norm", "B": 1, "T": 16384, "C": 4096, "dtype": "bf16",
         "residual": "bf16", "train": False, "bits8": True},
        # odd rows of odd width
        {"name": "norm_24x999x999_f16", "kind": "norm", "B": 24, "T": 999, "C": 999, "dtype": "f16",
         "residual": "f16", "train": True, "bits8": False},
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    kind = rng.choice(["conv_step", "conv", "conv", "scan_step", "scan", "scan", "scan", "norm", "norm"])
    dtype = rng.choice(["f32", "f16", "bf16"])
    if kind == "conv_step":
        return {"kind": kind, "B": _log(rng, 1, 512), "C": _log(rng, 64, 4097), "K": rng.randint(2, 4), "dtype": dtype}
    if kind == "scan_step":
        G = rng.choice([1, 1, 2])
        return {"kind": kind, "B": _log(rng, 1, 512), "D": G * _log(rng, 64, 2049), "N": rng.choice([4, 8, 16, 16]),
                "G": G, "dtype": dtype}
    T = _log(rng, 1, 100000)
    C = _log(rng, 16, 4100)
    if kind == "norm":
        T = max(1, min(T, (1 << 26) // C))
        B = max(1, min(_log(rng, 1, 32), (1 << 26) // (C * T)))
        train = rng.random() < 0.6
        return {"kind": kind, "B": B, "T": T, "C": C, "dtype": dtype, "residual": rng.choice([dtype, "f32", "none"]),
                "train": train, "bits8": not train and rng.random() < 0.6}
    if kind == "conv":
        T = max(1, min(T, (1 << 26) // C))
        B = max(1, min(_log(rng, 1, 32), (1 << 26) // (C * T)))
        return {"kind": kind, "B": B, "T": T, "C": C, "K": rng.randint(2, 4), "dtype": dtype,
                "train": rng.random() < 0.6, "packed": rng.random() < 0.5, "state": rng.random() < 0.5,
                "ragged": rng.random() < 0.4}
    G = rng.choice([1, 1, 1, 2, 4])
    N = rng.choice([4, 8, 16, 16, 16, 24, 32, 64])
    D = max(G, C // G * G)
    T = max(1, min(T, (1 << 29) // (D * N)))
    B = max(1, min(_log(rng, 1, 32), (1 << 29) // (D * N * T)))
    return {"kind": kind, "B": B, "T": T, "D": D, "N": N, "G": G, "dtype": dtype, "train": rng.random() < 0.6,
            "gate": rng.random() < 0.7, "skip": rng.random() < 0.8, "bias": rng.random() < 0.8,
            "state": rng.random() < 0.5, "ragged": rng.random() < 0.4}


def _lengths(case, g):
    B, T = case["B"], case["T"]
    if not case["ragged"]:
        return None
    n = torch.randint(1, T + 1, (B,), generator=g, device="cuda")
    n[0] = T
    if B > 1:
        n[B // 2] = 0
    return n.to(torch.int32)


def _dynamics(s, D, N, g):
    """The parameters of a scan: steps of 0.001 to 0.1 at dt = 0, decay rates around 1..N."""
    step = torch.exp(torch.empty(D, device="cuda").uniform_(math.log(1e-3), math.log(1e-1), generator=g))
    s["dt_bias"] = torch.log(torch.expm1(step))
    rate = torch.arange(1, N + 1, device="cuda").float().log().repeat(D, 1)
    s["a_log"] = rate + 0.1 * torch.randn(D, N, generator=g, device="cuda")
    s["d"] = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")


def prepare(case, seed):
    dev = "cuda"
    g = torch.Generator(device=dev)
    g.manual_seed(seed)
    td = DTYPES[case["dtype"]]

    def randn(*shape, dtype=torch.float32):
        return torch.randn(*shape, generator=g, device=dev).to(dtype)

    s = dict(case)
    kind = case["kind"]
    if kind == "norm":
        shape = (case["B"], case["T"], case["C"])
        s["x"] = randn(*shape, dtype=td)
        s["w"] = 1 + 0.1 * randn(case["C"])
        s["res"] = None if case["residual"] == "none" else randn(*shape, dtype=DTYPES[case["residual"]])
        if case["train"]:
            s["dy"] = randn(*shape, dtype=td)
            s["dtotal"] = None if s["res"] is None else randn(*shape, dtype=s["res"].dtype)
        return s
    if kind in ("conv", "conv_step"):
        B, C, K = case["B"], case["C"], case["K"]
        s["w"] = (torch.rand(C, K, generator=g, device=dev) * 2 - 1) / math.sqrt(K)
        s["bias"] = (torch.rand(C, generator=g, device=dev) * 2 - 1) / math.sqrt(K)
        if kind == "conv_step":
            s["x"] = randn(B, 2 * C, dtype=td).chunk(2, dim=1)[0]  # half of the projection
            slots = B + B // 4 + 1
            s["cache"] = randn(slots, K - 1, C, dtype=td)
            s["slots"] = torch.randperm(slots, generator=g, device=dev)[:B].to(torch.int32)
            return s
        T = case["T"]
        s["proj"] = randn(B, T, 2 * C, dtype=td) if case["packed"] else None
        s["x"] = s["proj"].chunk(2, dim=2)[0] if case["packed"] else randn(B, T, C, dtype=td)
        s["h0"] = randn(B, K - 1, C, dtype=td) if case["state"] else None
        s["lengths"] = _lengths(case, g)
        if case["train"]:
            s["dy"] = randn(B, T, C, dtype=td)
            s["dlast"] = randn(B, K - 1, C, dtype=td) if case["state"] else None
        return s
    B, D, N, G = case["B"], case["D"], case["N"], case["G"]
    _dynamics(s, D, N, g)
    rank = max(1, D // 16)
    if kind == "scan_step":
        s["x"], s["dt"] = randn(B, D, dtype=td), (0.5 * randn(B, D)).to(td)
        s["z"] = randn(B, 2 * D, dtype=td).chunk(2, dim=1)[1]
        low = randn(B, rank + 2 * G * N, dtype=td)  # dt's low-rank factor, b and c come from one projection
        s["b"], s["c"] = low[:, rank:rank + G * N], low[:, rank + G * N:]
        slots = B + B // 4 + 1
        s["cache"] = 0.1 * randn(slots, D, N)
        s["slots"] = torch.randperm(slots, generator=g, device=dev)[:B].to(torch.int32)
        return s
    T = case["T"]
    s["x"], s["dt"] = randn(B, T, D, dtype=td), (0.5 * randn(B, T, D)).to(td)
    s["z"] = randn(B, T, 2 * D, dtype=td).chunk(2, dim=2)[1] if case["gate"] else None
    s["rank"] = rank
    low = randn(B, T, rank + 2 * G * N, dtype=td)
    s["b"], s["c"] = low[..., rank:rank + G * N], low[..., rank + G * N:]
    if not case["skip"]:
        s["d"] = None
    if not case["bias"]:
        s["dt_bias"], s["dt"] = None, (s["dt"].float() - 4).to(td)
    s["h0"] = 0.1 * randn(B, D, N) if case["state"] else None
    s["lengths"] = _lengths(case, g)
    if case["train"]:
        s["dy"] = randn(B, T, D, dtype=td)
        s["dh_last"] = randn(B, D, N) if case["state"] else None
    return s


# ---------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------

def _silu(v):
    return v * torch.sigmoid(v)


def _dsilu(v):
    k = torch.sigmoid(v)
    return k * (1 + v * (1 - k))


def _live(s):
    """[B, T, 1]: the positions that count."""
    return torch.arange(s["T"], device="cuda").view(1, -1, 1) < s["lengths"].view(-1, 1, 1)


def _plain_norm(s):
    td = DTYPES[s["dtype"]]
    total = s["x"].float()
    if s["res"] is not None:
        total = (total + s["res"].float()).to(s["res"].dtype)
    v = total.float()
    rstd = torch.rsqrt(v.square().mean(-1, keepdim=True) + EPS)
    n = v * rstd
    y = n * s["w"]
    out = {} if s["res"] is None else {"total": total}
    if s["bits8"]:
        scale = y.abs().amax(-1) / TOP
        k = torch.where(scale > 0, 1 / scale, 0.0)
        out["y"] = (y * k.unsqueeze(-1)).clamp(-TOP, TOP).to(torch.float8_e4m3fn)
        out["scale"] = scale
        return out
    out["y"] = y.to(td)
    if not s["train"]:
        return out
    dy = s["dy"].float()
    g = dy * s["w"]
    ds = rstd * (g - n * (g * n).mean(-1, keepdim=True))
    if s["dtotal"] is not None:
        ds = ds + s["dtotal"].float()
    out["dx"] = ds.to(td)
    if s["res"] is not None and s["res"].dtype != td:
        out["dresidual"] = ds.to(s["res"].dtype)
    out["dw"] = (dy * n).sum((0, 1))
    return out


def _plain_conv(s):
    td, K, T = DTYPES[s["dtype"]], s["K"], s["T"]
    x = s["x"].float()
    B, C = x.shape[0], x.shape[2]
    live = None if s["lengths"] is None else _live(s)
    h0 = torch.zeros(B, K - 1, C, device="cuda") if s["h0"] is None else s["h0"].float()
    win = torch.cat([h0, x], 1).unfold(1, K, 1)  # [B, T, C, K]
    v = (win * s["w"]).sum(-1) + s["bias"]
    y = _silu(v)
    n = torch.full((B,), T, device="cuda") if live is None else s["lengths"].long()
    at = n.view(-1, 1) + torch.arange(K - 1, device="cuda")  # rows of [h0, x] that the state holds
    rows = at.unsqueeze(-1).expand(-1, -1, C)
    out = {"y": (y if live is None else torch.where(live, y, 0.0)).to(td),
           "last": torch.cat([h0, x], 1).gather(1, rows).to(td)}
    if not s["train"]:
        return out
    dv = s["dy"].float() * _dsilu(v)
    if live is not None:
        dv = torch.where(live, dv, 0.0)
    # what reaches row j of [h0, x]: sum_k w[k] dv[j - k]
    d = torch.nn.functional.pad(dv, (0, 0, K - 1, K - 1)).unfold(1, K, 1)  # [B, T + K - 1, C, K]
    d = (d * s["w"].flip(1)).sum(-1)
    if s["dlast"] is not None:
        d = d.scatter_add(1, rows, s["dlast"].float())
    dx = d[:, K - 1:]
    out["dx"] = (dx if live is None else torch.where(live, dx, 0.0)).to(td)
    out["dw"] = (win * dv.unsqueeze(-1)).sum((0, 1)) if live is None else \
        (torch.where(live.unsqueeze(-1), win, 0.0) * dv.unsqueeze(-1)).sum((0, 1))
    out["dbias"] = dv.sum((0, 1))
    if s["h0"] is not None:
        out["dh0"] = d[:, :K - 1].to(td)
    return out


def _plain_conv_step(s):
    at = s["slots"].long()
    win = torch.cat([s["cache"][at], s["x"].unsqueeze(1)], 1)
    v = (win.float() * s["w"].t()).sum(1) + s["bias"]
    s["cache"][at] = win[:, 1:]
    return {"y": _silu(v).to(DTYPES[s["dtype"]]), "cache": s["cache"]}


def _scan(a, b):
    """Inclusive scan of h_t = a_t h_{t-1} + b_t over axis 1, by doubling."""
    T, reach = a.shape[1], 1
    while reach < T:  # log2(T) passes: a recurrence has no elementwise form
        b = torch.cat([b[:, :reach], torch.addcmul(b[:, reach:], a[:, reach:], b[:, :-reach])], 1)
        a = torch.cat([a[:, :reach], a[:, reach:] * a[:, :-reach]], 1)
        reach *= 2
    return b


def _channels(s, t):
    """b or c, [..., G * N], for every channel: [..., D, N]."""
    G, N = s["G"], s["N"]
    return t.float().unflatten(-1, (G, N)).repeat_interleave(s["D"] // G, -2)


def _groups(s, t):
    """The sum of [..., D, N] over the channels of a group, [..., G * N]."""
    return t.unflatten(-2, (s["G"], s["D"] // s["G"])).sum(-2).flatten(-2)


def _plain_sscan(s):
    td, N = DTYPES[s["dtype"]], s["N"]
    x, dt = s["x"].float(), s["dt"].float()
    B, T, D = x.shape
    live = None if s["lengths"] is None else _live(s)
    if s["dt_bias"] is not None:
        dt = dt + s["dt_bias"]
    delta = torch.nn.functional.softplus(dt)
    if live is not None:
        delta = torch.where(live, delta, 0.0)
        x = torch.where(live, x, 0.0)
    A = -torch.exp(s["a_log"])
    b, c = _channels(s, s["b"]), _channels(s, s["c"])
    a = torch.exp(delta.unsqueeze(-1) * A)
    u = (delta * x).unsqueeze(-1)
    h0 = torch.zeros(B, D, N, device="cuda") if s["h0"] is None else s["h0"]
    put = u * b
    if live is not None:
        put = torch.where(live.unsqueeze(-1), put, 0.0)
    put[:, 0] += a[:, 0] * h0
    h = _scan(a, put)
    del put
    sums = (h * c).sum(-1)
    if s["d"] is not None:
        sums = sums + s["d"] * x
    z = None if s["z"] is None else s["z"].float()
    y = sums if z is None else sums * _silu(z)
    out = {"y": (y if live is None else torch.where(live, y, 0.0)).to(td), "h_last": h[:, -1].clone()}
    if not s["train"]:
        return out
    dy = s["dy"].float()
    if live is not None:
        dy = torch.where(live, dy, 0.0)
    ds = dy if z is None else dy * _silu(z)
    dz = None if z is None else dy * sums * _dsilu(z)
    del sums
    come = ds.unsqueeze(-1) * c
    if live is not None:
        come = torch.where(live.unsqueeze(-1), come, 0.0)
    if s["dh_last"] is not None:
        come[:, -1] += s["dh_last"]
    after = torch.cat([a[:, 1:], torch.ones_like(a[:, :1])], 1)
    gr = _scan(after.flip(1), come.flip(1)).flip(1)
    del after, come
    db, dc = _groups(s, gr * u), _groups(s, ds.unsqueeze(-1) * h)
    q = gr * a * torch.cat([h0.unsqueeze(1), h[:, :-1]], 1)
    gb = gr * b
    if live is not None:  # what lies behind a sequence is not looked at
        dz = None if dz is None else torch.where(live, dz, 0.0)
        db, dc = torch.where(live, db, 0.0), torch.where(live, dc, 0.0)
        gb = torch.where(live.unsqueeze(-1), gb, 0.0)
    gb = gb.sum(-1)
    dx = delta * gb
    ddt = ((q * A).sum(-1) + x * gb) * torch.sigmoid(dt)
    if live is not None:
        ddt = torch.where(live, ddt, 0.0)
    if s["d"] is not None:
        dx = dx + ds * s["d"]
        out["dd"] = (ds * x).sum((0, 1))
    out["dx"], out["ddt"] = dx.to(td), ddt.to(td)
    out["db"], out["dc"] = db.to(td), dc.to(td)
    out["da_log"] = (q * delta.unsqueeze(-1)).sum((0, 1)) * A
    if z is not None:
        out["dz"] = dz.to(td)
    if s["dt_bias"] is not None:
        out["ddt_bias"] = ddt.sum((0, 1))
    if s["h0"] is not None:
        out["dh0"] = a[:, 0] * gr[:, 0]
    return out


def _plain_sscan_step(s):
    at = s["slots"].long()
    x = s["x"].float()
    delta = torch.nn.functional.softplus(s["dt"].float() + s["dt_bias"])
    a = torch.exp(delta.unsqueeze(-1) * -torch.exp(s["a_log"]))
    h = a * s["cache"][at] + (delta * x).unsqueeze(-1) * _channels(s, s["b"])
    s["cache"][at] = h
    sums = (h * _channels(s, s["c"])).sum(-1) + s["d"] * x
    return {"y": (sums * _silu(s["z"].float())).to(DTYPES[s["dtype"]]), "cache": s["cache"]}


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

PLAIN = {"norm": _plain_norm, "conv": _plain_conv, "conv_step": _plain_conv_step, "scan": _plain_sscan,
         "scan_step": _plain_sscan_step}


def run(state):
    if not own:
        return PLAIN[state["kind"]](state)
    import aware_conv_amd
    return {"norm": _own_norm, "conv": _own_conv, "conv_step": _own_conv_step, "scan": _own_sscan,
            "scan_step": _own_sscan_step}[state["kind"]](aware_conv_amd, state)


def _own_norm(A, s):
    if s["bits8"]:
        y, scale, total = A.rmsnorm_fwd_e4m3(s["x"], s["w"], residual=s["res"], eps=EPS)
        return {"y": y, "scale": scale, "total": total}
    y, total, rstd = A.rmsnorm_fwd(s["x"], s["w"], residual=s["res"], eps=EPS, save_rstd=s["train"])
    out = {"y": y, "total": total}
    if s["train"]:
        kept = s["x"] if total is None else total
        g = A.rmsnorm_bwd(kept, s["w"], rstd, s["dy"], dtotal=s["dtotal"])
        out["dx"], out["dw"] = g["dx"], g["dw"]
        if s["res"] is not None and s["res"].dtype != s["x"].dtype:
            out["dresidual"] = g["dresidual"]
    return out


def _own_conv(A, s):
    y, last = A.cconv_fwd(s["x"], s["w"], bias=s["bias"], h0=s["h0"], lengths=s["lengths"], silu=True)
    out = {"y": y, "last": last}
    if s["train"]:
        grads = None
        if s["proj"] is not None:  # its half of the projection's gradient
            grads = {"dx": torch.empty_like(s["proj"]).chunk(2, dim=2)[0]}
        g = A.cconv_bwd(s["x"], s["w"], s["dy"], bias=s["bias"], h0=s["h0"], dlast=s["dlast"], lengths=s["lengths"],
                        silu=True, grads=grads)
        out.update({k: g[k] for k in ("dx", "dw", "dbias")})
        if s["h0"] is not None:
            out["dh0"] = g["dh0"]
    return out


def _own_conv_step(A, s):
    y = A.cconv_step(s["x"], s["w"], s["cache"], bias=s["bias"], slots=s["slots"], silu=True)
    return {"y": y, "cache": s["cache"]}


def _own_sscan(A, s):
    form = {"d": s["d"], "z": s["z"], "dt_bias": s["dt_bias"], "lengths": s["lengths"]}
    y, h_last, states = A.sscan_fwd(s["x"], s["dt"], s["a_log"], s["b"], s["c"], h0=s["h0"], save_states=s["train"],
                                    **form)
    out = {"y": y, "h_last": h_last}
    if s["train"]:
        # b, c and z are parts of projections, and so are their gradients
        B, T, D = s["x"].shape
        n, r = s["G"] * s["N"], s["rank"]
        low = torch.empty(B, T, r + 2 * n, dtype=y.dtype, device=y.device)
        grads = {"db": low[..., r:r + n], "dc": low[..., r + n:]}
        if s["z"] is not None:
            grads["dz"] = torch.empty(B, T, 2 * D, dtype=y.dtype, device=y.device).chunk(2, dim=2)[1]
        g = A.sscan_bwd(s["x"], s["dt"], s["a_log"], s["b"], s["c"], states, s["dy"], dh_last=s["dh_last"],
                        grads=grads, **form)
        out.update({k: v for k, v in g.items() if k != "dh0" or s["h0"] is not None})
    return out


def _own_sscan_step(A, s):
    y = A.sscan_step(s["x"], s["dt"], s["a_log"], s["b"], s["c"], s["cache"], d=s["d"], z=s["z"],
                     dt_bias=s["dt_bias"], slots=s["slots"])
    return {"y": y, "cache": s["cache"]}


def work(case):
    e, B = SIZES[case["dtype"]], case["B"]
    if case["kind"] == "norm":
        n = B * case["T"] * case["C"]
        r = 0 if case["residual"] == "none" else SIZES[case["residual"]]
        y = 1 if case["bits8"] else e
        if not case["train"]:
            return {"bytes": n * (e + 2 * r + y) + 4 * case["C"], "flops": 6 * n}
        two = r if r and r != e else 0  # the residual's gradient, where it is another tensor than x's
        return {"bytes": n * (4 * e + 3 * r + two) + 8 * case["C"], "flops": 16 * n}
    if case["kind"] == "conv_step":
        n, K = B * case["C"], case["K"]
        return {"bytes": n * e * 2 * K + 4 * case["C"] * (K + 1), "flops": n * (2 * K + 5)}
    if case["kind"] == "conv":
        n, K = B * case["T"] * case["C"], case["K"]
        small = 4 * case["C"] * (K + 1) + B * (K - 1) * case["C"] * e * (1 + case["state"])
        if not case["train"]:
            return {"bytes": 2 * n * e + small, "flops": n * (2 * K + 5)}
        return {"bytes": 4 * n * e + 2 * small, "flops": n * (6 * K + 15)}
    D, N, G = case["D"], case["N"], case["G"]
    if case["kind"] == "scan_step":
        return {"bytes": B * D * (4 * e + 8 * N) + 2 * B * G * N * e + 4 * D * (N + 2), "flops": B * D * (7 * N + 20)}
    n, low = B * case["T"] * D, B * case["T"] * G * N
    small = 4 * B * D * N * (1 + case["state"]) + 4 * D * (N + 2)
    if not case["train"]:
        return {"bytes": n * e * (3 + case["gate"]) + 2 * low * e + small, "flops": n * (7 * N + 20)}
    return {"bytes": n * e * (6 + 2 * case["gate"]) + 4 * low * e + 2 * small, "flops": n * (26 * N + 60)}


# ---------------------------------------------------------------------------
# from the definitions, in 64 bits, one sequence after the other
# ---------------------------------------------------------------------------

def _exact_recurrence(a, b, first):
    """h_t = a_t h_{t-1} + b_t with h_{-1} = first over the first axis: the sequence is cut into pieces
    that advance together, then each piece is given the state it starts from."""
    T = a.shape[0]
    if T == 0:
        return b
    piece = max(1, int(math.sqrt(T)))
    count = -(-T // piece)
    fill = count * piece - T
    rest = a.shape[1:]
    a = torch.cat([a, a.new_ones(fill, *rest)]).view(count, piece, *rest)
    h = torch.cat([b, b.new_zeros(fill, *rest)]).view(count, piece, *rest)
    grown = torch.empty_like(a)
    grown[:, 0] = a[:, 0]
    for t in range(1, piece):
        h[:, t] += a[:, t] * h[:, t - 1]
        grown[:, t] = a[:, t] * grown[:, t - 1]
    start = first
    for k in range(count):
        h[k] += grown[k] * start
        start = h[k, -1]
    return h.view(count * piece, *rest)[:T]


def _exact_sscan(s):
    B, T, D, N, G = (s[k] for k in ("B", "T", "D", "N", "G"))
    lengths = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"y": zeros(B, T, D), "h_last": zeros(B, D, N)}
    if s["train"]:
        out.update({k: zeros(B, T, D) for k in ("dx", "ddt")})
        out.update({k: zeros(B, T, G * N) for k in ("db", "dc")})
        out.update({"da_log": zeros(D, N), "dd": zeros(D), "ddt_bias": zeros(D), "dz": zeros(B, T, D),
                    "dh0": zeros(B, D, N)})
    step = max(1, min(D // G, (1 << 27) // max(1, T * N)))  # channels at a time
    for i in range(B):
        n = lengths[i]
        for first in range(0, D, D // G):
            k = first // (D // G)
            b, c = (s[m][i, :n, k * N:(k + 1) * N].double()[:, None] for m in ("b", "c"))
            for lo in range(first, first + D // G, step):
                at = slice(lo, min(lo + step, first + D // G))
                x = s["x"][i, :n, at].double()
                pre = s["dt"][i, :n, at].double()
                if s["dt_bias"] is not None:
                    pre = pre + s["dt_bias"][at].double()
                delta = torch.logaddexp(pre, torch.zeros_like(pre))
                rate = torch.exp(s["a_log"][at].double())
                start = zeros(x.shape[1], N) if s["h0"] is None else s["h0"][i, at].double()
                a = torch.exp(-delta[..., None] * rate)
                h = _exact_recurrence(a, (delta * x)[..., None] * b, start)
                out["h_last"][i, at] = h[-1] if n else start
                v = (c * h).sum(-1)
                if s["d"] is not None:
                    v = v + s["d"][at].double() * x
                open_, way = 1.0, None
                if s["z"] is not None:
                    z = s["z"][i, :n, at].double()
                    way = 1 / (1 + torch.exp(-z))
                    open_ = z * way
                out["y"][i, :n, at] = v * open_
                if not s["train"]:
                    continue
                dy = s["dy"][i, :n, at].double()
                dv = dy * open_
                if way is not None:
                    out["dz"][i, :n, at] = dy * v * (way + z * way * (1 - way))
                end = zeros(x.shape[1], N) if s["dh_last"] is None else s["dh_last"][i, at].double()
                # what goes back through position t: r_t = a_t (dv_t c_t + r_{t+1}), r_T = dh_last
                r = _exact_recurrence(a.flip(0), (a * dv[..., None] * c).flip(0), end).flip(0)
                gh = dv[..., None] * c + torch.cat([r[1:], end[None]])[:n]
                out["db"][i, :n, k * N:(k + 1) * N] += torch.bmm(gh.transpose(1, 2).contiguous(),
                                                                 (delta * x)[..., None])[..., 0]
                out["dc"][i, :n, k * N:(k + 1) * N] += torch.bmm(h.transpose(1, 2).contiguous(), dv[..., None])[..., 0]
                past = torch.cat([start[None], h])[:n]
                d_power = gh * a * past  # gradient of delta A
                d_delta = (gh * b).sum(-1) * x - (d_power * rate).sum(-1)
                out["da_log"][at] -= (d_power * delta[..., None]).sum(0) * rate
                d_pre = d_delta / (1 + torch.exp(-pre))
                out["ddt"][i, :n, at] = d_pre
                out["ddt_bias"][at] += d_pre.sum(0)
                d_x = (gh * b).sum(-1) * delta
                if s["d"] is not None:
                    d_x = d_x + dv * s["d"][at].double()
                    out["dd"][at] += (dv * x).sum(0)
                out["dx"][i, :n, at] = d_x
                out["dh0"][i, at] = r[0] if n else end
    for name, there in (("dd", "d"), ("ddt_bias", "dt_bias"), ("dz", "z"), ("dh0", "h0")):
        if s[there] is None:
            out.pop(name, None)
    return out


def _exact_conv(s):
    B, T, C, K = (s[k] for k in ("B", "T", "C", "K"))
    lengths = [T] * B if s["lengths"] is None else s["lengths"].tolist()
    zeros = lambda *shape: torch.zeros(*shape, dtype=torch.float64, device="cuda")  # noqa: E731
    out = {"y": zeros(B, T, C), "last": zeros(B, K - 1, C)}
    if s["train"]:
        out.update({"dx": zeros(B, T, C), "dw": zeros(C, K), "dbias": zeros(C), "dh0": zeros(B, K - 1, C)})
    w, bias = s["w"].double(), s["bias"].double()
    for i in range(B):
        n = lengths[i]
        before = zeros(K - 1, C) if s["h0"] is None else s["h0"][i].double()
        line = torch.cat([before, s["x"][i, :n].double()])
        v = sum(line[k:k + n] * w[:, k] for k in range(K)) + bias
        way = 1 / (1 + torch.exp(-v))
        out["y"][i, :n] = v * way
        out["last"][i] = line[n:]
        if not s["train"]:
            continue
        dv = s["dy"][i, :n].double() * (way + v * way * (1 - way))
        d = torch.zeros_like(line)
        for k in range(K):
            d[k:k + n] += dv * w[:, k]
            out["dw"][:, k] += (dv * line[k:k + n]).sum(0)
        if s["dlast"] is not None:
            d[n:] += s["dlast"][i].double()
        out["dbias"] += dv.sum(0)
        out["dx"][i, :n], out["dh0"][i] = d[K - 1:], d[:K - 1]
    if s["h0"] is None:
        out.pop("dh0", None)
    return out


def _exact_norm(s):
    total = s["x"].double()
    if s["res"] is not None:
        # the sum is rounded to the residual's type, and that is what is normed
        total = (total + s["res"].double()).to(s["res"].dtype).double()
    inv = 1 / torch.sqrt((total * total).sum(-1, keepdim=True) / s["C"] + EPS)
    w = s["w"].double()
    y = total * inv * w
    out = {} if s["res"] is None else {"total": total}
    if s["bits8"]:
        size = y.abs().max(-1).values / TOP
        x = torch.where(size[..., None] > 0, y / size[..., None], 0)
        fine = torch.ldexp(torch.ones_like(x), (torch.frexp(x.abs()).exponent - 1).clamp(min=-6) - 3)
        out["y"], out["scale"] = torch.round(x / fine) * fine, size
        return out
    out["y"] = y
    if s["train"]:
        dy = s["dy"].double()
        g = dy * w
        d = inv * g - total * inv ** 3 * (g * total).sum(-1, keepdim=True) / s["C"]
        if s["dtotal"] is not None:
            d = d + s["dtotal"].double()
        out["dx"] = d
        if s["res"] is not None and s["res"].dtype != s["x"].dtype:
            out["dresidual"] = d
        out["dw"] = (dy * total * inv).sum((0, 1))
    return out


def exact(case, seed):
    s = prepare(case, seed)
    if s["kind"] == "norm":
        return _exact_norm(s)
    if s["kind"] == "conv":
        return _exact_conv(s)
    if s["kind"] == "scan":
        return _exact_sscan(s)
    at = s["slots"].long()
    cache = s["cache"].double()
    x = s["x"].double()
    if s["kind"] == "conv_step":
        line = torch.cat([cache[at], x[:, None]], 1)
        v = torch.stack([line[:, k] * s["w"][:, k].double() for k in range(s["K"])]).sum(0) + s["bias"].double()
        cache[at] = line[:, 1:]
        return {"y": v / (1 + torch.exp(-v)), "cache": cache}
    G, N, D = s["G"], s["N"], s["D"]
    pre = s["dt"].double() + s["dt_bias"].double()
    delta = torch.logaddexp(pre, torch.zeros_like(pre))[..., None]
    group = torch.arange(D, device=x.device) // (D // G)
    b, c = (s[m].double().view(-1, G, N)[:, group] for m in ("b", "c"))
    h = torch.exp(-delta * torch.exp(s["a_log"].double())) * cache[at] + delta * x[..., None] * b
    cache[at] = h
    z = s["z"].double()
    return {"y": ((c * h).sum(-1) + s["d"].double() * x) * z / (1 + torch.exp(-z)), "cache": cache}
