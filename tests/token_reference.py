"""The selective scan, the causal convolution and the root-mean-square norm from their formulas in
fp64 on the CPU, one position after the other: what the tests of the kernels compare with.  Where
an output sums terms of both signs, the sum of their magnitudes is returned too (`mass`)."""
import torch


def sig(v):
    return 1 / (1 + torch.exp(-v))


def silu(v):
    return v * sig(v)


def dsilu(v):
    return sig(v) * (1 + v * (1 - sig(v)))


def softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp_min(0)


def counts(B, T, lengths):
    return [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths]


def _spread(low, D, N):
    """b or c [T, G * N] for each channel, [T, D, N]."""
    G = low.shape[-1] // N
    return low.unflatten(-1, (G, N)).repeat_interleave(D // G, 1)


def _gather(t, G):
    """[T, D, N] summed over the channels of a group, [T, G * N]."""
    return t.unflatten(1, (G, t.shape[1] // G)).sum(2).flatten(1)


def sscan(x, dt, a_log, b, c, d=None, z=None, dt_bias=None, h0=None, lengths=None, dy=None, dh_last=None):
    """Outputs (and, with dy, gradients) by name, and their masses."""
    B, T, D = x.shape
    N = a_log.shape[1]
    G = b.shape[-1] // N
    A = -torch.exp(a_log)
    zero = torch.zeros
    f64 = {"dtype": torch.float64}
    out = {"y": zero(B, T, D, **f64), "h_last": zero(B, D, N, **f64) if h0 is None else h0.clone()}
    mass = {"y": zero(B, T, D, **f64)}
    if dy is not None:
        for k in ("dx", "ddt", "dz"):
            out[k], mass[k] = zero(B, T, D, **f64), zero(B, T, D, **f64)
        for k in ("db", "dc"):
            out[k], mass[k] = zero(B, T, G * N, **f64), zero(B, T, G * N, **f64)
        for k, n in (("da_log", (D, N)), ("dd", (D,)), ("ddt_bias", (D,))):
            out[k], mass[k] = zero(*n, **f64), zero(*n, **f64)
        out["dh0"] = zero(B, D, N, **f64)
    for i, n in enumerate(counts(B, T, lengths)):
        pre = dt[i, :n] + (0 if dt_bias is None else dt_bias)
        delta = softplus(pre)
        a = torch.exp(delta[..., None] * A)
        u = delta * x[i, :n]
        bb, cc = _spread(b[i, :n], D, N), _spread(c[i, :n], D, N)
        h = out["h_last"][i].clone()
        before, after = zero(n, D, N, **f64), zero(n, D, N, **f64)
        for t in range(n):
            before[t] = h
            h = a[t] * h + u[t][:, None] * bb[t]
            after[t] = h
        out["h_last"][i] = h
        dk = zero(D, **f64) if d is None else d
        s = (cc * after).sum(-1) + dk * x[i, :n]
        s_mass = (cc * after).abs().sum(-1) + (dk * x[i, :n]).abs()
        gate = torch.ones(n, D, **f64) if z is None else silu(z[i, :n])
        out["y"][i, :n], mass["y"][i, :n] = s * gate, s_mass * gate.abs()
        if dy is None:
            continue
        ds = dy[i, :n] * gate
        if z is not None:
            out["dz"][i, :n] = dy[i, :n] * s * dsilu(z[i, :n])
            mass["dz"][i, :n] = (dy[i, :n] * s_mass * dsilu(z[i, :n])).abs()
        r = zero(D, N, **f64) if dh_last is None else dh_last[i].clone()
        g = zero(n, D, N, **f64)
        for t in range(n)[::-1]:
            g[t] = ds[t][:, None] * cc[t] + r
            r = a[t] * g[t]
        out["dh0"][i] = r
        q = g * a * before
        gb = g * bb
        out["db"][i, :n], mass["db"][i, :n] = _gather(g * u[..., None], G), _gather((g * u[..., None]).abs(), G)
        t = ds[..., None] * after
        out["dc"][i, :n], mass["dc"][i, :n] = _gather(t, G), _gather(t.abs(), G)
        out["dx"][i, :n] = delta * gb.sum(-1) + dk * ds
        mass["dx"][i, :n] = delta * gb.abs().sum(-1) + (dk * ds).abs()
        ddt = ((A * q).sum(-1) + x[i, :n] * gb.sum(-1)) * sig(pre)
        m = ((A * q).abs().sum(-1) + x[i, :n].abs() * gb.abs().sum(-1)) * sig(pre)
        out["ddt"][i, :n], mass["ddt"][i, :n] = ddt, m
        out["ddt_bias"] += ddt.sum(0)
        mass["ddt_bias"] += m.sum(0)
        out["da_log"] += (delta[..., None] * q).sum(0) * A
        mass["da_log"] -= (delta[..., None] * q).abs().sum(0) * A
        out["dd"] += (ds * x[i, :n]).sum(0)
        mass["dd"] += (ds * x[i, :n]).abs().sum(0)
    return out, mass


def cconv(x, w, bias=None, h0=None, lengths=None, act=True, dy=None, dlast=None):
    B, T, C = x.shape
    K = w.shape[1]
    f64 = {"dtype": torch.float64}
    out = {"y": torch.zeros(B, T, C, **f64), "last": torch.zeros(B, K - 1, C, **f64)}
    mass = {"y": torch.zeros(B, T, C, **f64)}
    if dy is not None:
        out.update(dx=torch.zeros(B, T, C, **f64), dw=torch.zeros(C, K, **f64), dbias=torch.zeros(C, **f64),
                   dh0=torch.zeros(B, K - 1, C, **f64))
        mass.update({k: torch.zeros_like(out[k]) for k in ("dx", "dw", "dbias", "dh0")})
    for i, n in enumerate(counts(B, T, lengths)):
        line = torch.cat([torch.zeros(K - 1, C, **f64) if h0 is None else h0[i], x[i, :n]])
        out["last"][i] = line[n:]
        v = torch.zeros(n, C, **f64) if bias is None else bias.expand(n, C).clone()
        m = v.abs()
        for k in range(K):
            v += w[:, k] * line[k:k + n]
            m = m + (w[:, k] * line[k:k + n]).abs()
        out["y"][i, :n] = silu(v) if act else v
        mass["y"][i, :n] = m * 1.1  # silu's slope is below 1.1
        if dy is None:
            continue
        dv = dy[i, :n] * (dsilu(v) if act else 1)
        # the slope moves by at most half of what v is off
        off = dy[i, :n].abs() * (1.1 + 0.5 * m if act else 1)
        d, dm = torch.zeros_like(line), torch.zeros_like(line)
        for k in range(K):
            d[k:k + n] += w[:, k] * dv
            dm[k:k + n] += w[:, k].abs() * off
            out["dw"][:, k] += (dv * line[k:k + n]).sum(0)
            mass["dw"][:, k] += (off * line[k:k + n].abs()).sum(0)
        out["dbias"] += dv.sum(0)
        mass["dbias"] += off.sum(0)
        if dlast is not None:
            d[n:] += dlast[i]
            dm[n:] += dlast[i].abs()
        out["dx"][i, :n], out["dh0"][i] = d[K - 1:], d[:K - 1]
        mass["dx"][i, :n], mass["dh0"][i] = dm[K - 1:], dm[:K - 1]
    return out, mass


def rmsnorm(total, w, eps, dy=None, dtotal=None):
    """From the sum that is normed (already rounded)."""
    rstd = 1 / torch.sqrt((total ** 2).mean(-1, keepdim=True) + eps)
    n = total * rstd
    out, mass = {"y": n * w, "rstd": rstd[..., 0]}, {}
    if dy is not None:
        g = dy * w
        mean = (g * n).mean(-1, keepdim=True)
        out["dx"] = rstd * (g - n * mean) + (0 if dtotal is None else dtotal)
        mass["dx"] = rstd * (g.abs() + n.abs() * (g * n).abs().mean(-1, keepdim=True)) + (
            0 if dtotal is None else dtotal.abs())
        out["dw"] = (dy * n).flatten(0, -2).sum(0)
        mass["dw"] = (dy * n).abs().flatten(0, -2).sum(0)
    return out, mass


def e4m3(y):
    """The e4m3 values nearest to y (ties to even), |y| <= 448."""
    fine = torch.ldexp(torch.ones_like(y), (torch.frexp(y.abs()).exponent - 1).clamp(min=-6) - 3)
    return torch.round(y / fine) * fine
