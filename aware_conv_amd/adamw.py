"""Binding of the AdamW step over many tensors (include/adamw.h) and an
optimizer over it.

Moments are fp32, or ``torch.float8_e4m3fn`` codes of m and sqrt(v) with one
fp32 scale per BLOCK elements.  The step's number, the gradient norm and, where
given as tensors, the learning rate and the gradient scale stay on the device:
a step neither synchronises nor copies, and can be captured into a graph.
"""
import ctypes
import operator

import numpy as np
import torch

from . import _lib
from .gscan import _raw_stream

DTYPES = {torch.float32: 0, torch.float16: 1, torch.bfloat16: 2}
BLOCK = 256
CODES = torch.float8_e4m3fn


def _dtype_code(dtype):
    if dtype not in DTYPES:
        raise TypeError("AdamW supports float32, float16 and bfloat16 parameters, got %s" % dtype)
    return DTYPES[dtype]


# Lists of tensors are checked attribute by attribute, with maps over the
# attributes' own getters: a step over a hundred small tensors takes about as
# long on the host as on the GPU, and this is most of it.
_dtypes = operator.attrgetter("dtype")
_numel, _contiguous = torch.Tensor.numel, torch.Tensor.is_contiguous
_device, _address = torch.Tensor.get_device, torch.Tensor.data_ptr


def _check_list(name, ts, count, dtype, device, numels):
    """Every tensor of the list: of `dtype`, on `device`, contiguous, of its number of elements."""
    if len(ts) != count:
        raise ValueError("%s holds %d tensors, expected %d" % (name, len(ts), count))
    if not all(issubclass(c, torch.Tensor) for c in set(map(type, ts))):
        raise TypeError("%s must hold tensors" % name)
    if set(map(_dtypes, ts)) != {dtype}:
        raise TypeError("%s must hold %s tensors" % (name, dtype))
    if set(map(_device, ts)) != {device.index}:
        raise ValueError("%s must lie on %s" % (name, device))
    if not all(map(_contiguous, ts)):
        raise ValueError("%s must be contiguous" % name)
    if numels is not None and list(map(_numel, ts)) != numels:
        raise ValueError("%s have sizes %s, expected %s" % (name, list(map(_numel, ts)), numels))


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


def _table(columns, numels):
    """Host array of adamw_tensor: `columns` are lists of tensors, or None."""
    t = np.zeros((len(numels), 8), dtype=np.int64)
    for k, ts in enumerate(columns):
        if ts is not None:
            t[:, k] = np.fromiter(map(_address, ts), np.int64, len(ts))
    t[:, 7] = numels
    return t


def _workspace(table, device, workspace):
    if workspace is None:
        n = ctypes.c_size_t(0)
        _lib._check(_lib.lib.adamw_workspace_size(table.ctypes.data, len(table), ctypes.byref(n)),
                    "adamw_workspace_size")
        workspace = torch.empty(n.value, dtype=torch.uint8, device=device)
    elif not workspace.is_contiguous() or workspace.device != device:
        raise ValueError("workspace must be contiguous and on %s" % device)
    return workspace, workspace.numel() * workspace.element_size()


def adamw_grad_norm(grads, grad_scale=1.0, norm=None, workspace=None, stream=None):
    """2-norm of ``grad_scale`` times all gradients together, as one fp32 on the device."""
    grads = list(grads)
    if not grads:
        raise ValueError("adamw_grad_norm needs at least one gradient")
    device = _gpu_of("grads", grads)
    code = _dtype_code(grads[0].dtype)
    _check_list("grads", grads, len(grads), grads[0].dtype, device, None)
    scale, scale_dev = _scalar("grad_scale", grad_scale, device)
    if norm is None:
        norm = torch.empty(1, dtype=torch.float32, device=device)
    else:
        _scalar("norm", norm, device)
    table = _table([None, grads], list(map(_numel, grads)))
    ws, nws = _workspace(table, device, workspace)
    p = _lib._ptr
    _lib._check(_lib.lib.adamw_grad_norm(code, table.ctypes.data, len(table), scale, p(scale_dev),
                                         p(norm), p(ws), nws, _raw_stream(stream, device)),
                "adamw_grad_norm")
    return norm


def adamw_step(params, grads, exp_avgs, exp_avg_sqs, step, lr=1e-3, betas=(0.9, 0.999), eps=1e-8,
               weight_decay=0.01, masters=None, scales=None, grad_scale=1.0, grad_norm=None,
               max_norm=None, workspace=None, stream=None):
    """One AdamW step over lists of tensors, in place.

    step: int32 on the device, the steps taken so far (advanced).  masters: fp32 copies of the
    parameters, which are then what is updated.  scales: (of exp_avgs, of exp_avg_sqs), lists of
    fp32 tensors, where the moments are e4m3 codes (exp_avg_sqs of sqrt(v)); without it they are
    fp32.  grad_norm: what adamw_grad_norm gave, for max_norm, and to leave out a step whose norm
    is not finite.  lr and grad_scale may be one-element fp32 tensors on the device."""
    params = list(params)
    if not params:
        return
    device = _gpu_of("params", params)
    dtype, count = params[0].dtype, len(params)
    code = _dtype_code(dtype)
    numels = list(map(_numel, params))
    _check_list("params", params, count, dtype, device, None)
    _check_list("grads", grads, count, dtype, device, numels)
    state = CODES if scales is not None else torch.float32
    _check_list("exp_avgs", exp_avgs, count, state, device, numels)
    _check_list("exp_avg_sqs", exp_avg_sqs, count, state, device, numels)
    if masters is not None:
        _check_list("masters", masters, count, torch.float32, device, numels)
    ms = vs = None
    if scales is not None:
        ms, vs = scales
        blocks = [-(-n // BLOCK) for n in numels]
        _check_list("scales[0]", ms, count, torch.float32, device, blocks)
        _check_list("scales[1]", vs, count, torch.float32, device, blocks)
    _step(params, grads, exp_avgs, exp_avg_sqs, step, lr, betas, eps, weight_decay, masters,
          (ms, vs), numels, code, device, grad_scale, grad_norm, max_norm, workspace, stream)


def _step(params, grads, exp_avgs, exp_avg_sqs, step, lr, betas, eps, weight_decay, masters,
          scales, numels, code, device, grad_scale, grad_norm, max_norm, workspace=None, stream=None):
    """The call, for lists that were checked or are the optimizer's own."""
    ms, vs = scales
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
    table = _table([params, grads, masters, exp_avgs, exp_avg_sqs, ms, vs], numels)
    ws, nws = _workspace(table, device, workspace)
    p = _lib._ptr
    config = _lib.AdamwConfig(code, 8 if ms is not None else 32, lr, betas[0], betas[1], eps,
                              weight_decay, scale, max_norm or 0.0, p(lr_dev), p(scale_dev),
                              p(grad_norm))
    _lib._check(_lib.lib.adamw_step(ctypes.byref(config), table.ctypes.data, len(numels), p(step), p(ws),
                                    nws, _raw_stream(stream, device)), "adamw_step")


class AdamW(torch.optim.Optimizer):
    """AdamW over ``adamw_step``: the parameters of a group that have one dtype and have taken
    the same steps are stepped by one call, with their moments and their step number on the
    device.

    bits: 32 or 8, of the moments.  master: keep fp32 copies of 16-bit parameters.  max_norm:
    clip the norm of all gradients together.  skip_nonfinite (implied by max_norm): leave out
    steps whose norm is not finite, moments and step numbers included.  lr (of a group) and
    grad_scale (an attribute: 1 / the loss scale) may be fp32 tensors on the device."""

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

            device, dtype, count = _gpu_of("parameters", ps), ps[0].dtype, len(ps)
            numels = list(map(_numel, ps))
            _check_list("parameters", ps, count, dtype, device, None)
            _check_list("gradients", gs, count, dtype, device, numels)
            scales = column("exp_avg_scale"), column("exp_avg_sq_scale")
            _step(ps, gs, column("exp_avg"), column("exp_avg_sq"), step, group["lr"],
                  group["betas"], group["eps"], group["weight_decay"], column("master"), scales,
                  numels, _dtype_code(dtype), device, self.grad_scale, norm, self.max_norm)
        return loss
