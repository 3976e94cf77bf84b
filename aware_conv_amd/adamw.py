"""Binding of the AdamW step over many tensors (include/adamw.h) and an
optimizer over it.

Moments are fp32, or ``torch.float8_e4m3fn`` codes of m and sqrt(v) with one
fp32 scale per BLOCK elements.  The step's number, the gradient norm and, where
given as tensors, the learning rate and the gradient scale stay on the device:
a step neither synchronises nor copies, and can be captured into a graph.
"""
import ctypes
import math

import numpy as np
import torch

from . import _lib
from .gscan import _lists, _raw_stream, on_stream

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
BLOCK = 256
CODES = torch.float8_e4m3fn


def _dtype_code(dtype):
    if dtype not in DTYPES:
        raise TypeError("AdamW supports float32, float16 and bfloat16 parameters, got %s" % dtype)
    return DTYPES[dtype]


# Lists of tensors are checked, and their addresses written into the call's
# table, by a small extension (pyext/tensor_lists.cpp).
_PARAM, _GRAD, _MASTER, _M, _V, _M_SCALE, _V_SCALE, _COUNT = range(8)  # columns of the table


def _held(ts):
    """The tensors as a list or tuple.  The table takes their addresses alone: who fills it keeps
    this until the call was enqueued, or tensors that only an iterator made would be gone."""
    return ts if isinstance(ts, (list, tuple)) else list(ts)


def _column(table, at, column, name, ts, dtype, device, block=1):
    """The list's addresses into the table, which lies `at` its own, after checking that its
    tensors are of `dtype`, on `device`, contiguous, and of ceil(n / block) elements for the n of
    the table's last column (block 0: of any number, which that column then takes)."""
    code, k = _lists.column(ts, at, len(table), column, dtype, device.index, block)
    if code == 0:
        return
    if code == 1:
        raise ValueError("%s holds %d tensors, expected %d" % (name, len(ts), len(table)))
    if code == 2:
        raise TypeError("%s[%d] must be a torch.Tensor" % (name, k))
    t = ts[k]
    if code == 3:
        raise TypeError("%s[%d] has dtype %s, expected %s" % (name, k, t.dtype, dtype))
    if code == 4:
        raise ValueError("%s[%d] is on %s, expected %s" % (name, k, t.device, device))
    if code == 5:
        raise ValueError("%s[%d] must be contiguous" % (name, k))
    raise ValueError("%s[%d] has %d elements, expected %d"
                     % (name, k, t.numel(), -(-int(table[k, _COUNT]) // block)))


def _new_table(count):
    return np.zeros((count, 8), dtype=np.int64)


def _gpu_of(name, ts):
    if not isinstance(ts[0], torch.Tensor):
        raise TypeError("%s must hold tensors" % name)
    if ts[0].device.type != "cuda":
        raise ValueError("%s[0] is on %s; every tensor must be on a GPU" % (name, ts[0].device))
    return ts[0].device


def _scalar(name, v, device):
    """(host value, device tensor or None) of a number or a one-element fp32 tensor."""
    if isinstance(v, torch.Tensor):
        if v.numel() != 1 or v.dtype != torch.float32 or v.device != device:
            raise ValueError("%s must be a number or one float32 on %s" % (name, device))
        return 0.0, v
    return float(v), None


def _workspace(table, at, device, workspace):
    if workspace is None:
        n = ctypes.c_size_t(0)
        _lib._check(_lib.lib.adamw_workspace_size(at, len(table), ctypes.byref(n)),
                    "adamw_workspace_size")
        workspace = torch.empty(n.value, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("workspace must be contiguous and on %s" % device)
    return workspace, workspace.numel() * workspace.element_size()


@on_stream
def adamw_grad_norm(grads, grad_scale=1.0, norm=None, workspace=None, *, stream=None):
    """2-norm of ``grad_scale`` times all gradients together, as one fp32 on the device."""
    grads = _held(grads)
    if not grads:
        raise ValueError("adamw_grad_norm needs at least one gradient")
    device = _gpu_of("grads", grads)
    code = _dtype_code(grads[0].dtype)
    table = _new_table(len(grads))
    at = table.ctypes.data  # asked for once: numpy takes 1 us for it
    _column(table, at, _GRAD, "grads", grads, grads[0].dtype, device, 0)
    scale, scale_dev = _scalar("grad_scale", grad_scale, device)
    given = norm
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=device)
    else:
        _scalar("norm", norm, device)
    ws, nws = _workspace(table, at, device, workspace)
    p = _lib._ptr
    _lib._enqueue(device, "adamw_grad_norm", code, at, len(table), scale, p(scale_dev), p(norm),
                  p(ws), nws, _raw_stream(stream, device))
    _lists.written(given)
    return norm


@on_stream
def adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
               weight_decay=0.01, masters=None, scales=None, grad_scale=1.0, grad_norm=None,
               max_norm=None, workspace=None, *, stream=None):
    """One AdamW step over lists of tensors, in place.

    step: int32 on the device, the steps taken so far (advanced).  masters: fp32 copies of the
    parameters, which are then what is updated.  scales: (of exp_avgs, of exp_avg_sqs), lists of
    fp32 tensors, where the moments are e4m3 codes (exp_avg_sqs of sqrt(v)); without it they are
    fp32.  grad_norm: what adamw_grad_norm gave, for max_norm, and to leave out a step whose norm
    is not finite.  lr and grad_scale may be one-element fp32 tensors on the device."""
    params = _held(params)
    if not params:
        return
    grads, exp_avgs, exp_avg_sqs = _held(grads), _held(exp_avgs), _held(exp_avg_sqs)
    masters = None if masters is None else _held(masters)
    scales = None if scales is None else [_held(ts) for ts in scales]
    device = _gpu_of("params", params)
    dtype, code = params[0].dtype, _dtype_code(params[0].dtype)
    table = _new_table(len(params))
    at = table.ctypes.data
    _column(table, at, _PARAM, "params", params, dtype, device, 0)
    _column(table, at, _GRAD, "grads", grads, dtype, device)
    state = CODES if scales is not None else torch.float32
    _column(table, at, _M, "exp_avgs", exp_avgs, state, device)
    _column(table, at, _V, "exp_avg_sqs", exp_avg_sqs, state, device)
    if masters is not None:
        _column(table, at, _MASTER, "masters", masters, torch.float32, device)
    if scales is not None:
        _column(table, at, _M_SCALE, "scales[0]", scales[0], torch.float32, device, BLOCK)
        _column(table, at, _V_SCALE, "scales[1]", scales[1], torch.float32, device, BLOCK)
    if not isinstance(step, torch.Tensor) or step.dtype != torch.int32 or step.numel() != 1 or \
            step.device != device:
        raise ValueError("step must be one int32 on %s" % device)
    if max_norm is not None and grad_norm is None:
        raise ValueError("max_norm needs grad_norm")
    lr, lr_dev = _scalar("lr", lr, device)
    scale, scale_dev = _scalar("grad_scale", grad_scale, device)
    if grad_norm is not None:
        if not isinstance(grad_norm, torch.Tensor):
            raise TypeError("grad_norm must be a torch.Tensor")
        _scalar("grad_norm", grad_norm, device)
    ws, nws = _workspace(table, at, device, workspace)
    p = _lib._ptr
    config = _lib.AdamwConfig(code, 8 if scales is not None else 32, lr, betas[0], betas[1], eps,
                              weight_decay, scale, max_norm or 0.0, p(lr_dev), p(scale_dev),
                              p(grad_norm))
    _lib._enqueue(device, "adamw_step", ctypes.byref(config), at, len(table), p(step), p(ws), nws,
                  _raw_stream(stream, device))
    _lists.written(params, exp_avgs, exp_avg_sqs, masters, step, *(scales or ()))


class AdamW(torch.optim.Optimizer):
    """AdamW over ``adamw_step``: the parameters of a group that have one dtype and have taken
    the same steps are stepped by one call, with their moments and their step number on the
    device.

    bits: 32 or 8, of the moments.  master: keep fp32 copies of 16-bit parameters.  max_norm:
    clip the norm of all gradients together.  skip_nonfinite (implied by max_norm): leave out
    steps whose norm is not finite, moments and step numbers included.  lr (of a group) and
    grad_scale (an attribute: 1 / the loss scale) may be fp32 tensors on the device.

    Parameters are contiguous and, where steps are clipped or left out, all on one device."""

    _OPTIONS = ("bits", "master", "max_norm", "skip_nonfinite", "grad_scale")

    def __init__(self, params, lr=1e-3, betas=(0.9, 0.999), eps=1e-8, weight_decay=0.01, bits=32,
                 master=True, max_norm=None, skip_nonfinite=False, grad_scale=1.0):
        if bits not in (8, 32):
            raise ValueError("bits must be 8 or 32, got %r" % (bits,))
        if not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError("betas must lie in [0, 1), got %r" % (betas,))
        if max_norm is not None and not max_norm > 0:
            raise ValueError("max_norm must be positive, got %r" % (max_norm,))
        self.bits, self.master, self.max_norm = bits, master, max_norm
        self.skip_nonfinite, self.grad_scale = skip_nonfinite, grad_scale
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay))

    def __getstate__(self):  # of copies and pickles; the base class keeps its own attributes alone
        return dict(super().__getstate__(), **{n: getattr(self, n) for n in self._OPTIONS})

    def add_param_group(self, param_group):
        super().add_param_group(param_group)
        group, wrong = self.param_groups[-1], None
        for n in ("lr", "eps", "weight_decay"):
            v = group[n]
            if not isinstance(v, torch.Tensor) and not 0.0 <= v < math.inf:
                wrong = "%s must be finite and not negative, got %r" % (n, v)
        if not all(p.is_contiguous() for p in group["params"]):
            wrong = "parameters must be contiguous"
        if wrong:
            self.param_groups.pop()
            raise ValueError(wrong)

    def _new_state(self, p, step):
        if not p.is_contiguous():
            raise ValueError("parameters must be contiguous")
        s = {"step": step}
        for n in ("exp_avg", "exp_avg_sq"):
            if self.bits == 8:
                # code 0 is the value 0
                s[n] = torch.zeros(p.shape, dtype=torch.uint8, device=p.device).view(CODES)
                s[n + "_scale"] = torch.zeros(-(-p.numel() // BLOCK), device=p.device)
            else:
                s[n] = torch.zeros(p.shape, dtype=torch.float32, device=p.device)
        if self.master and p.dtype != torch.float32:
            s["master"] = p.detach().float()
        return s

    def load_state_dict(self, state_dict):
        """The states as they were saved (the base class would cast codes and masters to the
        parameter's dtype); parameters of a group with equal step numbers share them again."""
        super().load_state_dict(state_dict)
        saved = state_dict["state"]
        for group, old in zip(self.param_groups, state_dict["param_groups"]):
            shared = {}
            for p, k in zip(group["params"], old["params"]):
                if k not in saved:
                    continue
                s = {n: t.detach().to(p.device, copy=True) for n, t in saved[k].items()}
                s["step"] = shared.setdefault((p.dtype, p.device, int(s["step"])), s["step"])
                self.state[p] = s

    def _runs(self):
        """(group, parameters, step number) of each call."""
        runs = []
        for group in self.param_groups:
            users, by_step, new = {}, {}, {}
            for p in group["params"]:
                s = self.state.get(p)
                if s:
                    users[id(s["step"])] = users.get(id(s["step"]), 0) + 1
                if p.grad is None:
                    continue
                if s:
                    by_step.setdefault(id(s["step"]), []).append(p)
                else:
                    new.setdefault((p.dtype, p.device), []).append(p)
            for ps in new.values():
                step = torch.zeros(1, dtype=torch.int32, device=ps[0].device)
                for p in ps:
                    self.state[p] = self._new_state(p, step)
                runs.append((group, ps, step))
            for key, ps in by_step.items():
                step = self.state[ps[0]]["step"]
                if len(ps) < users[key]:  # the others stay behind
                    step = step.clone()
                    for p in ps:
                        self.state[p]["step"] = step
                runs.append((group, ps, step))
        return runs

    def _norm(self, grads):
        by_type = {}
        for g in grads:
            by_type.setdefault(g.dtype, []).append(g)
        norms = [adamw_grad_norm(gs, self.grad_scale) for gs in by_type.values()]
        return norms[0] if len(norms) == 1 else adamw_grad_norm(norms)

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        runs = self._runs()
        grads = [[p.grad.contiguous() for p in ps] for _, ps, _ in runs]
        norm = None
        if runs and (self.max_norm is not None or self.skip_nonfinite):
            norm = self._norm([g for gs in grads for g in gs])
        for (group, ps, step), gs in zip(runs, grads):
            st = [self.state[p] for p in ps]

            def column(name):
                return [s[name] for s in st] if name in st[0] else None

            scales = None
            if self.bits == 8:
                scales = column("exp_avg_scale"), column("exp_avg_sq_scale")
            adamw_step(ps, gs, column("exp_avg"), column("exp_avg_sq"), step, lr=group["lr"],
                       betas=group["betas"], eps=group["eps"], weight_decay=group["weight_decay"],
                       masters=column("master"), scales=scales, grad_scale=self.grad_scale,
                       grad_norm=norm, max_norm=self.max_norm)
        return loss
