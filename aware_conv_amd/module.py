"""torch.autograd and nn.Module wrappers over the C ABI."""
import math
import operator

import torch

from . import _lib, cconv, gscan, rmsnorm, sscan


class WTConvFunction(torch.autograd.Function):
    """Forward through ``wtconv_fwd``; backward through ``wtconv_bwd`` (input
    and parameter gradients from one pass), or the one of ``wtconv_bwd_input``
    and ``wtconv_bwd_weight`` that is needed.  Only x and the parameters are
    saved: the subband tensors are recomputed by the backward kernels."""

    @staticmethod
    def forward(ctx, x, w_base, b_base, s_base, w_wav, s_wav):
        ctx.save_for_backward(x, w_base, b_base, s_base, w_wav, s_wav)
        return _lib.wtconv_fwd(x, w_base, b_base, s_base, w_wav, s_wav)

    @staticmethod
    def backward(ctx, dy):
        x, w_base, b_base, s_base, w_wav, s_wav = ctx.saved_tensors
        dy = dy.contiguous()
        dx = None
        g = {n: None for n in _lib.GRAD_NAMES}
        want_dx, want_g = ctx.needs_input_grad[0], any(ctx.needs_input_grad[1:])
        if want_dx and want_g:
            dx, g = _lib.wtconv_bwd(x, dy, w_base, b_base, s_base, w_wav, s_wav)
        elif want_dx:
            dx = _lib.wtconv_bwd_input(dy, w_base, s_base, w_wav, s_wav)
        elif want_g:
            g = _lib.wtconv_bwd_weight(x, dy, w_base, b_base, s_base, w_wav, s_wav)
        return dx, g["dw_base"], g["db_base"], g["ds_base"], g["dw_wav"], g["ds_wav"]


class WTConv2d(torch.nn.Module):
    """Wavelet depthwise convolution with ``levels`` Haar levels and a
    ``kernel_size`` x ``kernel_size`` filter per channel and subband."""

    def __init__(self, channels, kernel_size=5, levels=2, base_scale=1.0,
                 wavelet_scale=0.1, device=None, dtype=None):
        super().__init__()
        f = {"device": device, "dtype": dtype}
        k, C, L = kernel_size, channels, levels
        self.w_base = torch.nn.Parameter(torch.empty(C, 1, k, k, **f))
        self.b_base = torch.nn.Parameter(torch.zeros(C, **f))
        self.s_base = torch.nn.Parameter(torch.full((C,), float(base_scale), **f))
        self.w_wav = torch.nn.Parameter(torch.empty(L, C, 4, k, k, **f))
        self.s_wav = torch.nn.Parameter(torch.full((L, C, 4), float(wavelet_scale), **f))
        with torch.no_grad():
            self.w_base.normal_(0, 0.02)
            self.w_wav.normal_(0, 0.02)

    def forward(self, x):
        return WTConvFunction.apply(x.contiguous(), self.w_base, self.b_base, self.s_base,
                                    self.w_wav, self.s_wav)


class GatedScan2d(torch.nn.Module):
    """Gated linear recurrence over whole planes [B, C, H, W] in raster order, its gates two
    WTConv layers of the input: each output mixes all positions before it (and, where ``both``,
    in a second recurrence from the end, all positions after it).

    lam is fp32 whatever the layer's dtype; at a fully open gate the decays start evenly spread
    over ``decay_range``."""

    DECAY = 8.0

    def __init__(self, channels, kernel_size=5, levels=2, both=True, decay_range=(0.9, 0.999),
                 device=None, dtype=None):
        super().__init__()
        f = {"device": device, "dtype": dtype}
        self.reset = WTConv2d(channels, kernel_size, levels, **f)
        self.input = WTConv2d(channels, kernel_size, levels, **f)
        lo, hi = decay_range
        a = torch.linspace(lo, hi, channels, dtype=torch.float64)
        lam = torch.log(torch.expm1(-torch.log(a) / self.DECAY)).float()
        self.lam = torch.nn.Parameter(lam.repeat(2 if both else 1, 1).to(device))
        self.scale = 1 / math.sqrt(2) if both else 1.0

    def _apply(self, fn, recurse=True):
        """Conversions of the layer (half(), to(dtype), ...) move lam and leave its dtype."""
        lam = [t for t in (self.lam, self.lam.grad) if t is not None]

        def converted(t):
            new = fn(t)
            return t.to(new.device) if any(t is k for k in lam) and new.dtype != t.dtype else new

        return super()._apply(converted, recurse)

    def forward(self, x):
        x = x.contiguous()
        r, i = self.reset(x), self.input(x)
        h = gscan.gated_scan(x, r, i, self.lam[0], decay=self.DECAY)[0]
        if len(self.lam) == 2:
            h = h + gscan.gated_scan(x, r, i, self.lam[1], reverse=True, decay=self.DECAY)[0]
        return h * self.scale


class SelectiveMixer(torch.nn.Module):
    """Block over token sequences [B, T, C]: the root-mean-square norm of the residual stream, a
    projection to twice ``expand * channels``, a short causal convolution and a selective state
    space scan of one half, gated by the other, and a projection back.

    ``forward`` takes the stream as the output x of the block before and what was added up before
    that (``residual``; None: x starts the stream), and returns its own output and the sum, to be
    handed on alike.  ``prompt`` also fills rows of a cache, from which ``step`` goes on one
    position at a time.

    Norm weight, convolution and the scan's parameters are fp32 whatever the layer's dtype; the
    steps start spread over ``step_range``, the decay rates at 1..states.

    Under autocast the projections and what follows them are in its dtype; the cache's rows keep
    the layer's (the convolution's inputs) and fp32 (the scan's states).

    A pass with its backward can be captured into a graph, as torch's own operations can: after a
    warm-up on another stream, and while no eager result of the same parameters that still holds
    its graph is alive (torch would draw that one's stream into the capture, and fail)."""

    _FP32 = ("norm", "conv_w", "conv_b", "dt_bias", "a_log", "d")

    def __init__(self, channels, states=16, expand=2, taps=4, rank=None, groups=1, eps=1e-5,
                 step_range=(1e-3, 1e-1), residual_fp32=False, device=None, dtype=None):
        super().__init__()
        f = {"device": device, "dtype": dtype}
        p = {"device": device, "dtype": torch.float32}
        inner = expand * channels
        rank = rank or max(1, channels // 16)
        self.split = (rank, groups * states, groups * states)
        self.eps, self.residual_fp32 = eps, residual_fp32
        self.inner = torch.nn.Linear(channels, 2 * inner, bias=False, **f)
        self.low = torch.nn.Linear(inner, sum(self.split), bias=False, **f)
        self.dt = torch.nn.Linear(rank, inner, bias=False, **f)
        self.outer = torch.nn.Linear(inner, channels, bias=False, **f)
        self.norm = torch.nn.Parameter(torch.ones(channels, **p))
        self.conv_w = torch.nn.Parameter(torch.empty(inner, taps, **p).uniform_(-1, 1) / math.sqrt(taps))
        self.conv_b = torch.nn.Parameter(torch.zeros(inner, **p))
        lo, hi = (math.log(s) for s in step_range)
        step = torch.exp(torch.linspace(lo, hi, inner, dtype=torch.float64))
        self.dt_bias = torch.nn.Parameter(torch.log(torch.expm1(step)).float().to(device))
        rate = torch.arange(1, states + 1, dtype=torch.float32).log()
        self.a_log = torch.nn.Parameter(rate.repeat(inner, 1).to(device))
        self.d = torch.nn.Parameter(torch.ones(inner, **p))

    def _apply(self, fn, recurse=True):
        """Conversions of the layer (half(), to(dtype), ...) move the parameters that stay in fp32
        and leave their dtype."""
        own = [t for n in self._FP32 for t in (getattr(self, n), getattr(self, n).grad) if t is not None]

        def converted(t):
            new = fn(t)
            return t.to(new.device) if any(t is k for k in own) and new.dtype != t.dtype else new

        return super()._apply(converted, recurse)

    def _stream(self, x, residual):
        """The residual that the norm adds x to: in fp32 from the block that starts the stream on."""
        if residual is None and self.residual_fp32:
            return torch.zeros_like(x, dtype=torch.float32)
        return residual

    def _mix(self, x, residual, lengths, conv0=None, h0=None):
        """(output, stream, the convolution's last inputs, the scan's last state)"""
        y, total = rmsnorm.rms_norm(x, self.norm, self._stream(x, residual), self.eps)
        u, z = self.inner(y).chunk(2, dim=-1)
        conv0 = None if conv0 is None else conv0.to(u.dtype)
        u, last = cconv.causal_conv(u, self.conv_w, self.conv_b, h0=conv0, lengths=lengths)
        dt, b, c = self.low(u).split(self.split, dim=-1)
        v, h = sscan.selective_scan(u, self.dt(dt), self.a_log, b, c, self.d, z, self.dt_bias, h0, lengths)
        return self.outer(v), x if total is None else total, last, h

    def forward(self, x, residual=None, lengths=None):
        """(output, residual stream) of x [B, T, C]; lengths [B] int32 where sequences are padded
        (with finite values where gradients are wanted: the projections see them)."""
        return self._mix(x, residual, lengths)[:2]

    def new_cache(self, rows):
        """Zeroed rows for ``prompt`` and ``step``: the convolution's inputs and the scan's states."""
        inner, taps = self.conv_w.shape
        f = {"device": self.a_log.device}
        return (torch.zeros(rows, taps - 1, inner, dtype=self.inner.weight.dtype, **f),
                torch.zeros(rows, inner, self.a_log.shape[1], **f))

    @torch.no_grad()
    def prompt(self, x, cache, residual=None, lengths=None, rows=None):
        """``forward`` from what rows of the cache hold (``rows``: their numbers, a list of integers;
        the first B if None), which then hold what ``step`` goes on from."""
        conv, state = cache
        rows = list(range(x.shape[0])) if rows is None else [operator.index(k) for k in rows]
        if len(rows) != x.shape[0] or len(set(rows)) != len(rows) or not all(0 <= k < len(state) for k in rows):
            raise ValueError("rows must be %d different rows of the cache's %d, got %s"
                             % (x.shape[0], len(state), rows))
        at = torch.tensor(rows, dtype=torch.long, device=state.device)
        out, total, last, state[at] = self._mix(x, residual, lengths, conv[at], state[at])
        conv[at] = last.to(conv.dtype)
        return out, total

    @torch.no_grad()
    def step(self, x, cache, residual=None, slots=None):
        """(output, residual stream) of one position x [B, C], which moves the cache's rows on."""
        y, total, _ = rmsnorm.rmsnorm_fwd(x, self.norm, residual=self._stream(x, residual), eps=self.eps)
        u, z = self.inner(y).chunk(2, dim=-1)
        u = cconv.cconv_step(u.to(cache[0].dtype), self.conv_w, cache[0], bias=self.conv_b, slots=slots).to(z.dtype)
        dt, b, c = self.low(u).split(self.split, dim=-1)
        v = sscan.sscan_step(u, self.dt(dt), self.a_log, b, c, cache[1], d=self.d, z=z, dt_bias=self.dt_bias,
                             slots=slots)
        return self.outer(v), x if total is None else total
