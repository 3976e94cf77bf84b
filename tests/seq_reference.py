"""The gated linear recurrence and the AdamW step from their formulas in fp64
on the CPU, one position (one element) after the other in the plainest way:
what the tests of the kernels compare with."""
import math

import numpy as np
import torch


def sig(v):
    return 1 / (1 + torch.exp(-v))


def softplus(v):
    return torch.log1p(torch.exp(-v.abs())) + v.clamp_min(0)


def orders(B, T, lengths, reverse):
    """For each sequence the valid positions in scan order."""
    n = [T] * B if lengths is None else [min(max(int(v), 0), T) for v in lengths]
    return [list(range(k))[::-1] if reverse else list(range(k)) for k in n]


def gates(x, r, i, lam, decay):
    L = -decay * softplus(lam) * sig(r)
    a = torch.exp(L)
    w = torch.sqrt(-torch.expm1(2 * L))
    return L, a, w, w * sig(i) * x


def fwd(x, r, i, lam, h0=None, lengths=None, reverse=False, decay=8.0):
    """x, r, i: [B, C, T] fp64.  Returns h, h_last and the state before each position."""
    B, C, T = x.shape
    _, a, _, b = gates(x, r, i, lam[None, :, None], decay)
    h, before = torch.zeros_like(x), torch.zeros_like(x)
    last = torch.zeros(B, C, dtype=x.dtype) if h0 is None else h0.clone()
    for n, order in enumerate(orders(B, T, lengths, reverse)):
        s = last[n].clone()
        for t in order:
            before[n, :, t] = s
            s = a[n, :, t] * s + b[n, :, t]
            h[n, :, t] = s
        last[n] = s
    return h, last, before


def bwd(x, r, i, lam, dh, h0=None, dh_last=None, lengths=None, reverse=False, decay=8.0):
    """Gradients, and under "mass" the sum of the magnitudes that dlam sums."""
    B, C, T = x.shape
    l3 = lam[None, :, None]
    L, a, w, _ = gates(x, r, i, l3, decay)
    _, _, before = fwd(x, r, i, lam, h0, lengths, reverse, decay)
    dx, dr, di, e = (torch.zeros_like(x) for _ in range(4))
    dh0 = torch.zeros(B, C, dtype=x.dtype) if dh_last is None else dh_last.clone()
    for n, order in enumerate(orders(B, T, lengths, reverse)):
        u = dh0[n].clone()
        for t in reversed(order):
            g = dh[n, :, t] + u
            si = sig(i[n, :, t])
            dx[n, :, t] = g * w[n, :, t] * si
            di[n, :, t] = dx[n, :, t] * x[n, :, t] * sig(-i[n, :, t])
            ratio = torch.where(w[n, :, t] > 0, a[n, :, t] ** 2 / w[n, :, t], 0.0)
            d = g * (a[n, :, t] * before[n, :, t] - si * x[n, :, t] * ratio)
            dr[n, :, t] = d * L[n, :, t] * sig(-r[n, :, t])
            e[n, :, t] = -d * sig(r[n, :, t])
            u = a[n, :, t] * g
        dh0[n] = u
    k = decay * sig(lam)
    return {"dx": dx, "dr": dr, "di": di, "dlam": k * e.sum((0, 2)), "dh0": dh0,
            "mass": k * e.abs().sum((0, 2))}


# e4m3: the 127 magnitudes in order
CODE_VALUES = np.array([m / 8 * 2.0 ** -6 if e == 0 else (1 + m / 8) * 2.0 ** (e - 7)
                        for e in range(16) for m in range(8)][:127])


def dither(n, t, turn):
    k = np.arange(n, dtype=np.uint64)
    u = (k * 2654435769 + np.uint64(t * 3242174889 + turn)) & np.uint64(0xFFFFFFFF)
    return (u >> np.uint64(8)).astype(np.float64) / 2 ** 24


def encode(values, t, root, error):
    """(values the codes stand for, scales, where rounding is too close to call) of fp64 values
    in blocks of 256; `root`: sqrt(v), which keeps a code above 0 where it is above 0.  `error`:
    what each value may be off by in fp32 (the division by the scale adds 2^-22 of it)."""
    n = len(values)
    out, close = np.zeros(n), np.zeros(n, dtype=bool)
    scales = np.zeros(-(-n // 256))
    d = dither(n, t, 2 ** 31 if root else 0)
    for b in range(len(scales)):
        part = slice(b * 256, min(n, b * 256 + 256))
        v = values[part]
        scales[b] = np.abs(v).max() / 448
        if scales[b] < 2.0 ** -126:
            scales[b] = 0
            continue
        x = np.abs(v) / scales[b]
        lo = np.clip(np.searchsorted(CODE_VALUES, x, side="right") - 1, 0, 125)
        frac = (x - CODE_VALUES[lo]) / (CODE_VALUES[lo + 1] - CODE_VALUES[lo])
        up = frac + d[part] >= 1
        q = CODE_VALUES[lo + up]
        if root:
            q = np.where((x > 0) & (q == 0), 2.0 ** -9, q)
        out[part] = np.copysign(q, v) * scales[b]
        off = (x * 2.0 ** -22 + error[part] / scales[b]) / (CODE_VALUES[lo + 1] - CODE_VALUES[lo])
        off = off + 2.0 ** -20  # the sum with the dither
        close[part] = (np.abs(frac + d[part] - 1) < off) | (frac < off) | (frac > 1 - off)
    return out, scales, close


def adamw(p, g, m, v, t, lr, betas, eps, weight_decay):
    """New (p, m, v) of fp64 arrays at step t (counted from 1)."""
    b1, b2 = betas
    m = b1 * m + (1 - b1) * g
    v = b2 * v + (1 - b2) * g * g
    p = p - lr * weight_decay * p - lr * (m / (1 - b1 ** t)) / (np.sqrt(v / (1 - b2 ** t)) + eps)
    return p, m, v


def norm(grads):
    return math.sqrt(sum(float((g.astype(np.float64) ** 2).sum()) for g in grads))
