"""Operators on lists of tensors for training: the gradients' norm, clipping
by it, and the AdamW step with the clipping folded in.

Each call goes over the whole list in a few launches (the norm's pass and the
updating pass), whatever the number and sizes of the tensors, and returns
without reading anything back to the host.  Autograd sees what is updated as
changed in place, as by torch's optimizers.  ``AdamW`` is an optimizer over
``adamw_step_``.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Iterable, List, Optional, Sequence

import torch
from torch.autograd.graph import increment_version

from . import SLA_BF16, SLA_F16, SLA_F32, SLA_F64, SLA_OK, SlaError, _on, _ptr, _raw_stream, load

__all__ = ["AdamW", "adamw_step_", "clip_grad_norm_", "grad_norm", "sla_adamw", "sla_clip_grads",
           "sla_grad_norm", "sla_grad_workspace_bytes"]

_TYPES = {torch.float64: SLA_F64, torch.float32: SLA_F32, torch.float16: SLA_F16,
          torch.bfloat16: SLA_BF16}


class _Tensor(ctypes.Structure):
    _fields_ = [("grad", ctypes.c_void_p), ("param", ctypes.c_void_p),
                ("exp_avg", ctypes.c_void_p), ("exp_avg_sq", ctypes.c_void_p),
                ("master", ctypes.c_void_p), ("n", ctypes.c_int64),
                ("step", ctypes.c_int64), ("grad_type", ctypes.c_int32),
                ("param_type", ctypes.c_int32), ("d_skipped", ctypes.c_void_p)]


# the structure as struct's native layout packs it
_PACK = struct.Struct("@5PqqiiP")


class _AdamOpts(ctypes.Structure):
    _fields_ = [("lr", ctypes.c_double), ("beta_one", ctypes.c_double),
                ("beta_two", ctypes.c_double), ("eps", ctypes.c_double),
                ("weight_decay", ctypes.c_double), ("max_norm", ctypes.c_double)]


# -------------------------------------------------------------- raw C calls

def sla_grad_workspace_bytes(count: int) -> int:
    return int(load().sla_grad_workspace_bytes(int(count)))


def sla_grad_norm(table, count, norm, work, stream) -> int:
    return load().sla_grad_norm(table, count, _ptr(norm), _TYPES[norm.dtype], _ptr(work), stream)


def sla_clip_grads(table, count, max_norm, norm, work, stream) -> int:
    return load().sla_clip_grads(table, count, float(max_norm), _ptr(norm), _TYPES[norm.dtype],
                                 _ptr(work), stream)


def sla_adamw(table, count, opts: _AdamOpts, norm, work, stream) -> int:
    return load().sla_adamw(table, count, ctypes.byref(opts), _ptr(norm),
                            _TYPES[norm.dtype] if norm is not None else SLA_F32, _ptr(work),
                            stream)


# ----------------------------------------------------------------- the lists

def _addresses(xs: Sequence[torch.Tensor], name: str, device: int) -> List[int]:
    """The addresses of dense tensors on the device."""
    if device < 0 or any(x.get_device() != device for x in xs):
        raise ValueError(f"{name} must be device tensors on one device")
    if not all(x.is_contiguous() for x in xs):
        raise ValueError(f"{name} must be contiguous")
    return [x.data_ptr() for x in xs]


def _types(xs: Sequence[torch.Tensor], what: str) -> List[int]:
    try:
        return [_TYPES[x.dtype] for x in xs]
    except KeyError as e:
        raise ValueError(f"{what} has dtype {e.args[0]}, expected float64, float32, float16 or "
                         "bfloat16") from None


def _table(rows) -> ctypes.Array:
    """An array of sla_tensor; rows give all members of one each."""
    rows = list(rows)
    table = (_Tensor * len(rows))()
    pack, size = _PACK.pack_into, _PACK.size
    for i, row in enumerate(rows):
        pack(table, i * size, *row)
    return table


def _grads_table(grads: Sequence[torch.Tensor], device: int) -> ctypes.Array:
    kinds = _types(grads, "a gradient")
    return _table((g, 0, 0, 0, 0, x.numel(), 1, kind, kind, 0)
                  for g, x, kind in zip(_addresses(grads, "gradients", device), grads, kinds))


def _norm_and_work(grads: Sequence[torch.Tensor], device):
    wide = any(g.dtype == torch.float64 for g in grads)
    norm = torch.empty((), dtype=torch.float64 if wide else torch.float32, device=device)
    return norm, torch.empty(sla_grad_workspace_bytes(len(grads)), dtype=torch.uint8,
                             device=device)


def _tensors(grads) -> List[torch.Tensor]:
    return [grads] if isinstance(grads, torch.Tensor) else list(grads)


def grad_norm(grads: Iterable[torch.Tensor], stream=None) -> torch.Tensor:
    """The 2-norm of all the tensors together, a scalar on their device:
    float64 if one of them is, else float32 (squares and sums are taken in
    fp64).  Tensors of any mix of float64, float32, float16 and bfloat16,
    contiguous.  A number about them: no gradient flows through it."""
    grads = _tensors(grads)
    if not grads:
        return torch.zeros((), device="cuda")
    device = grads[0].get_device()
    table = _grads_table(grads, device)
    with _on(device, stream):
        norm, work = _norm_and_work(grads, grads[0].device)
        st = sla_grad_norm(table, len(grads), norm, work, _raw_stream(norm))
    if st != SLA_OK:
        raise SlaError(st, "sla_grad_norm")
    return norm


def clip_grad_norm_(grads: Iterable[torch.Tensor], max_norm: float, stream=None) -> torch.Tensor:
    """Multiplies every tensor by min(1, max_norm / (norm + 1e-6)) in place
    and returns the norm before that (as ``grad_norm``).  Nothing is read to
    the host: a norm that is not finite shows in the returned scalar."""
    if not max_norm >= 0:
        raise ValueError("max_norm must not be negative")
    grads = _tensors(grads)
    if not grads:
        return torch.zeros((), device="cuda")
    device = grads[0].get_device()
    table = _grads_table(grads, device)
    with _on(device, stream):
        norm, work = _norm_and_work(grads, grads[0].device)
        st = sla_clip_grads(table, len(grads), max_norm, norm, work, _raw_stream(norm))
    if st != SLA_OK:
        raise SlaError(st, "sla_clip_grads")
    increment_version(grads)
    return norm


def adamw_step_(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
                exp_avgs: Sequence[torch.Tensor], exp_avg_sqs: Sequence[torch.Tensor], step,
                lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                weight_decay: float = 1e-2, max_norm: Optional[float] = None,
                masters: Optional[Sequence[Optional[torch.Tensor]]] = None, stream=None,
                skipped: Optional[Sequence[Optional[torch.Tensor]]] = None):
    """One AdamW step (decoupled weight decay) on every tensor, in place.

    ``step`` counts from 1: one number, or one for each tensor.  Moments are
    float64 for float64 params, else float32; float16 and bfloat16 params may
    have a float32 master each (``masters``, None where there is none), which
    the step then updates and the param is the rounding of.  Gradients have the
    param's type, or float32; float32 params also take float16 and bfloat16
    ones.  With ``max_norm`` the gradients are clipped to that global norm as
    they are read (they stay as they are) and the norm is returned; a norm that
    is not finite leaves everything as it is.  ``skipped`` counts such steps
    where the host does not see them: for each tensor an int64 scalar on the
    device (or None), raised by one when a step is skipped, and what it holds is
    taken off the tensor's ``step``."""
    n = len(params)
    masters = [None] * n if masters is None else masters
    steps = [step] * n if isinstance(step, int) else list(step)
    if not (len(steps) == len(grads) == len(exp_avgs) == len(exp_avg_sqs) == len(masters) == n):
        raise ValueError("params, grads, moments, masters and steps differ in number")
    if max_norm is not None and not max_norm > 0:
        raise ValueError("max_norm must be positive")
    if n == 0:
        return None if max_norm is None else torch.zeros((), device="cuda")
    device = params[0].get_device()
    kinds, grad_kinds = _types(params, "a param"), _types(grads, "a gradient")
    sizes = [g.numel() for g in grads]
    for p, g, m, v, w, n_g in zip(params, grads, exp_avgs, exp_avg_sqs, masters, sizes):
        pd, gd = p.dtype, g.dtype
        wide = torch.float64 if pd == torch.float64 else torch.float32
        if gd != pd and (gd == torch.float64 or wide == torch.float64 or
                         torch.float32 not in (gd, pd)):
            raise ValueError(f"a param of dtype {pd} with a gradient of {gd}")
        if not p.numel() == m.numel() == v.numel() == n_g:
            raise ValueError("a param, its gradient and its moments differ in size")
        if m.dtype != wide or v.dtype != wide:
            raise ValueError(f"the moments of a {pd} param must be {wide}")
        if w is not None and (pd in (torch.float32, torch.float64) or w.dtype != torch.float32 or
                              w.numel() != n_g):
            raise ValueError("a master is the float32 copy of a float16 or bfloat16 param")
    skipped = [None] * n if skipped is None else skipped
    counters = [x for x in skipped if x is not None]
    if len(skipped) != n or any(x.dtype != torch.int64 or x.numel() != 1 for x in counters):
        raise ValueError("skipped must hold an int64 scalar (or None) for each param")
    held = iter(_addresses([w for w in masters if w is not None], "masters", device))
    counters = iter(_addresses(counters, "counters", device))
    table = _table(zip(_addresses(grads, "gradients", device),
                       _addresses(params, "params", device),
                       _addresses(exp_avgs, "moments", device),
                       _addresses(exp_avg_sqs, "moments", device),
                       [0 if w is None else next(held) for w in masters], sizes, steps,
                       grad_kinds, kinds,
                       [0 if x is None else next(counters) for x in skipped]))
    with _on(device, stream):
        norm, work = _norm_and_work(grads, params[0].device) if max_norm is not None \
            else (None, None)
        opts = _AdamOpts(lr, betas[0], betas[1], eps, weight_decay, max_norm or 0.0)
        st = sla_adamw(table, n, opts, norm, work, _raw_stream(params[0]))
    if st != SLA_OK:
        raise SlaError(st, "sla_adamw")
    increment_version([*params, *exp_avgs, *exp_avg_sqs, *(w for w in masters if w is not None)])
    return norm


class AdamW(torch.optim.Optimizer):
    """AdamW over ``adamw_step_``: one norm pass and one updating pass for all
    parameters of a group.  ``max_norm`` clips each group's gradients to that
    norm within the step, every group by itself (``last_norm`` of the group holds
    its norm, on the device), and a step whose norm is not finite is skipped and
    does not count for the bias correction.  float16 and bfloat16 parameters get
    float32 masters.  Steps are counted on the host: a graph cannot capture them
    (``adamw_step_`` with a given step it can)."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8,
                 weight_decay: float = 1e-2, max_norm: Optional[float] = None):
        if lr < 0 or eps < 0 or not all(0 <= b < 1 for b in betas):
            raise ValueError("lr and eps must not be negative, betas must lie in [0, 1)")
        super().__init__(params, dict(lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                                      max_norm=max_norm))

    @torch.no_grad()
    def step(self, closure=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        for group in self.param_groups:
            params = [p for p in group["params"] if p.grad is not None]
            if any(not p.is_cuda for p in params):
                raise ValueError("params must be device tensors")
            if params and torch.cuda.is_current_stream_capturing():
                raise RuntimeError("AdamW.step counts steps on the host: it cannot be captured")
            for p in params:
                state = self.state[p]
                if not state:
                    wide = torch.float64 if p.dtype == torch.float64 else torch.float32
                    state["step"] = 0
                    state["exp_avg"] = torch.zeros_like(
                        p, dtype=wide, memory_format=torch.contiguous_format)
                    state["exp_avg_sq"] = torch.zeros_like(state["exp_avg"])
                    state["master"] = p.detach().float() if p.dtype in (
                        torch.float16, torch.bfloat16) else None
                if group["max_norm"] is not None and state.get("skipped") is None:
                    state["skipped"] = torch.zeros((), dtype=torch.int64, device=p.device)
            if not params:
                continue
            get = lambda name: [self.state[p][name] for p in params]
            group["last_norm"] = adamw_step_(
                params, [p.grad for p in params], get("exp_avg"), get("exp_avg_sq"),
                [n + 1 for n in get("step")], lr=group["lr"], betas=group["betas"],
                eps=group["eps"], weight_decay=group["weight_decay"],
                max_norm=group["max_norm"], masters=get("master"),
                skipped=[self.state[p].get("skipped") for p in params])
            for p in params:
                self.state[p]["step"] += 1
        return loss

    def state_dict(self):
        """Without the groups' ``last_norm``, which is an answer and no state."""
        saved = super().state_dict()
        for group in saved["param_groups"]:
            group.pop("last_norm", None)
        return saved

    def load_state_dict(self, state_dict):
        """Moments and masters keep their own types (the base class casts
        them to the parameters')."""
        super().load_state_dict(state_dict)
        kept = state_dict["state"]
        order = [p for group in self.param_groups for p in group["params"]]
        names = [i for group in state_dict["param_groups"] for i in group["params"]]
        for p, i in zip(order, names):
            for name, x in kept.get(i, {}).items():
                if isinstance(x, torch.Tensor):
                    self.state[p][name] = x.detach().clone().to(p.device)
