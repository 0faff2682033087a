"""The gated delta rule: a differentiable row-action solve over a sequence.

With the state S [dk, dv] of one head and a_t = exp(gate_t),

    w_t = v_t - a_t S_{t-1}^T k_t
    S_t = a_t S_{t-1} + beta_t k_t w_t^T
    o_t = scale S_t^T q_t

For unit keys, beta = 1 and gate = 0 each token projects S on its row of the
dense system k_t^T S = v_t (a Kaczmarz sweep); beta relaxes the projection
and the gate damps what was learnt before.  ``delta_rule`` takes whole
sequences (in chunks of 64 tokens, each a unit lower triangular solve) and
carries gradients, whose chunks are the transposed solves;
``delta_rule_step`` takes one token of many sequences and updates their
states in place.
"""
from __future__ import annotations

import ctypes
import struct
from typing import Optional, Tuple

import torch
from torch.autograd import forward_ad
from torch.autograd.graph import increment_version

from . import SLA_BF16, SLA_F16, SLA_F32, SLA_OK, SlaError, _on, _raw_stream, load

__all__ = ["DeltaRule", "delta_rule", "delta_rule_step", "sla_delta_forward",
           "sla_delta_backward", "sla_delta_step", "sla_delta_workspace_bytes",
           "sla_delta_saved_bytes"]

_TYPES = {torch.float32: SLA_F32, torch.float16: SLA_F16, torch.bfloat16: SLA_BF16}
MAX_DK = 128
_MAX_STRIDE = 1 << 22      # elements between the rows of v and o of neighbouring tokens


class _Args(ctypes.Structure):
    _fields_ = [("batch", ctypes.c_int64), ("tokens", ctypes.c_int64),
                ("key_heads", ctypes.c_int32), ("value_heads", ctypes.c_int32),
                ("dk", ctypes.c_int32), ("dv", ctypes.c_int32), ("dtype", ctypes.c_int32),
                ("scale", ctypes.c_float), ("d_q", ctypes.c_void_p), ("d_k", ctypes.c_void_p),
                ("d_v", ctypes.c_void_p), ("d_beta", ctypes.c_void_p),
                ("d_gate", ctypes.c_void_p), ("q_stride", ctypes.c_int64 * 3),
                ("k_stride", ctypes.c_int64 * 3), ("v_stride", ctypes.c_int64 * 3),
                ("beta_stride", ctypes.c_int64 * 3), ("gate_stride", ctypes.c_int64 * 3),
                ("d_lengths", ctypes.c_void_p)]


# the structure as struct's native layout packs it: one call fills all members
_PACK = struct.Struct("@qqiiiiif5P15qP")


# -------------------------------------------------------------- raw C calls

def sla_delta_workspace_bytes(args: _Args, backward: bool = False) -> int:
    return load().sla_delta_workspace_bytes(ctypes.byref(args), 1 if backward else 0)


def sla_delta_saved_bytes(args: _Args) -> int:
    return load().sla_delta_saved_bytes(ctypes.byref(args))


def _at(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def sla_delta_forward(args, state_in, state_out, o, o_stride, saved, work, stream) -> int:
    return load().sla_delta_forward(ctypes.byref(args), _at(state_in), _at(state_out), _at(o),
                                    o_stride, _at(saved), _at(work), work.numel(), stream)


def sla_delta_backward(args, saved, grad_o, o_stride, grad_state, dq, dk, dv, dbeta, dgate,
                       dstate, work, stream) -> int:
    return load().sla_delta_backward(ctypes.byref(args), _at(saved), _at(grad_o), o_stride,
                                     _at(grad_state), _at(dq), _at(dk), _at(dv), _at(dbeta),
                                     _at(dgate), _at(dstate), _at(work), work.numel(), stream)


def sla_delta_step(args, state, slots, o, o_stride, stream) -> int:
    return load().sla_delta_step(ctypes.byref(args), state.data_ptr(), state.shape[0], _at(slots),
                                 o.data_ptr(), o_stride, stream)


# ------------------------------------------------------------ argument checks

def _need(ok: bool, text: str):
    if not ok:
        raise ValueError(text)


def _like(x: torch.Tensor, name: str, shape, dtype, device: int):
    if not isinstance(x, torch.Tensor) or x.get_device() != device:
        raise ValueError(f"{name} must be a device tensor on device {device}")
    if x.shape != shape:
        raise ValueError(f"{name} has shape {tuple(x.shape)}, expected {tuple(shape)}")
    if x.dtype != dtype:
        raise ValueError(f"{name} has dtype {x.dtype}, expected {dtype}")


def _check_rule(q, k, v, beta, gate, state, lengths, lead: int) -> int:
    """Checks the arguments of a call whose tensors have ``lead`` leading
    dimensions before the heads' (2: batch and tokens; 1: batch); the device's index."""
    if not isinstance(v, torch.Tensor) or not v.is_cuda:
        raise ValueError("v must be a device tensor")
    device, vs, qs = v.get_device(), v.shape, q.shape
    if len(vs) != lead + 2 or len(qs) != lead + 2:
        raise ValueError(f"q and v must have {lead + 2} dimensions")
    if v.dtype not in _TYPES:
        raise ValueError(f"v has dtype {v.dtype}, expected float32, float16 or bfloat16")
    Hv, dv = vs[-2:]
    Hk, dk = qs[-2:]
    if Hk < 1 or Hv < 1 or Hv % Hk:
        raise ValueError(f"{Hv} value heads are not a multiple of {Hk} key heads")
    if not 1 <= dk <= MAX_DK:
        raise ValueError(f"key size {dk} is not in 1..{MAX_DK}")
    _need(dv >= 1, "values must have at least one column")
    _need(max(Hv * dv, Hk * dk) <= _MAX_STRIDE, "heads times their size exceed 2^22")
    keys, steps = vs[:lead] + qs[lead:], vs[:-1]
    _like(q, "q", keys, v.dtype, device)
    _like(k, "k", keys, v.dtype, device)
    _like(beta, "beta", steps, torch.float32, device)
    _like(gate, "gate", steps, torch.float32, device)
    if state is not None:
        _like(state, "state", (vs[0], Hv, dk, dv), torch.float32, device)
    if lengths is not None:
        _like(lengths, "lengths", (vs[0],), torch.int32, device)
        _need(lengths.is_contiguous(), "lengths must be contiguous")
    return device


def _rows(x: torch.Tensor, tokens: bool = False) -> torch.Tensor:
    """x, or a contiguous copy where the last dimension is not contiguous or
    (``tokens``) rows of neighbouring tokens overlap or lie too far apart."""
    shape, stride = x.shape, x.stride()
    dense = shape[-1] == 1 or stride[-1] == 1
    if tokens and shape[1] > 1:
        dense = dense and shape[-1] <= stride[1] <= _MAX_STRIDE
    return x if dense else x.contiguous()


_Stride = ctypes.c_int64 * 3


def _stride(x: torch.Tensor, tokens: bool = True):
    s = x.stride()
    return _Stride(s[0], s[1], s[2]) if tokens else _Stride(s[0], 0, s[1])


def _make_args(q, k, v, beta, gate, scale, lengths, tokens: bool = True) -> _Args:
    vs, qs = v.shape, q.shape
    strides = [q.stride(), k.stride(), v.stride(), beta.stride(), gate.stride()]
    if tokens:
        flat = [n for s in strides for n in s[:3]]
    else:
        flat = [n for s in strides for n in (s[0], 0, s[1])]
    args = _Args()
    _PACK.pack_into(args, 0, vs[0], vs[1] if tokens else 1, qs[-2], vs[-2], qs[-1], vs[-1],
                    _TYPES[v.dtype], scale, q.data_ptr(), k.data_ptr(), v.data_ptr(),
                    beta.data_ptr(), gate.data_ptr(), *flat,
                    0 if lengths is None else lengths.data_ptr())
    return args


def _in_dual_level() -> bool:
    """Whether tensors may carry forward-mode tangents (also with gradients off)."""
    return forward_ad._current_level >= 0


def _tracked(*xs) -> bool:
    """Whether a derivative of a result by one of the tensors is asked for."""
    return (torch.is_grad_enabled() and any(x.requires_grad for x in xs)) or (
        _in_dual_level() and any(forward_ad.unpack_dual(x).tangent is not None for x in xs))


def _bytes(n: int, device) -> torch.Tensor:
    return torch.empty(n, dtype=torch.uint8, device=device)


# ----------------------------------------------------------------- operators

def _forward(q, k, v, beta, gate, state, scale, lengths, save: bool):
    args = _make_args(q, k, v, beta, gate, scale, lengths)
    o = torch.empty(v.shape, dtype=v.dtype, device=v.device)
    last = torch.empty((v.shape[0], v.shape[2], q.shape[3], v.shape[3]), device=v.device)
    saved = _bytes(sla_delta_saved_bytes(args), v.device) if save else None
    work = _bytes(sla_delta_workspace_bytes(args), v.device)
    start = None if state is None else state.contiguous()
    st = sla_delta_forward(args, start, last, o, _stride(o), saved, work, _raw_stream(v))
    if st != SLA_OK:
        raise SlaError(st, "sla_delta_forward")
    return o, last, saved


class DeltaRule(torch.autograd.Function):
    """(o, last state) of ``delta_rule``'s arguments, checked as there; saves
    the inputs but v, the state at every chunk's start and W (4 (dk / 64 + 1) dv
    bytes a token and value head, dk and dv padded to whole tiles)."""

    @staticmethod
    def forward(ctx, q, k, v, beta, gate, state, scale, lengths):
        with _on(_check_rule(q, k, v, beta, gate, state, lengths, 2)):
            q, k, v = _rows(q), _rows(k), _rows(v, tokens=True)
            scale = q.shape[-1] ** -0.5 if scale is None else float(scale)
            o, last, saved = _forward(q, k, v, beta, gate, state, scale, lengths,
                                      any(ctx.needs_input_grad))
        if saved is not None:
            ctx.save_for_backward(q, k, beta, gate, lengths, saved)
            ctx.scale, ctx.has_state, ctx.dv = scale, state is not None, v.shape[3]
            ctx.set_materialize_grads(False)
        return o, last

    @staticmethod
    @torch.autograd.function.once_differentiable
    def backward(ctx, grad_o, grad_last):
        q, k, beta, gate, lengths, saved = ctx.saved_tensors
        new = lambda x: torch.empty(x.shape, dtype=x.dtype, device=x.device)
        dq, dk, dbeta, dgate = new(q), new(k), new(beta), new(gate)
        dv = torch.empty((*beta.shape, ctx.dv), dtype=q.dtype, device=q.device)
        grad_o = torch.zeros_like(dv) if grad_o is None else _rows(grad_o, tokens=True)
        grad_last = None if grad_last is None else grad_last.contiguous()
        dstate = torch.empty((q.shape[0], beta.shape[2], q.shape[3], ctx.dv),
                             device=q.device) if ctx.has_state else None
        # dv in v's place: of the shape and type, and not read
        args = _make_args(q, k, dv, beta, gate, ctx.scale, lengths)
        work = _bytes(sla_delta_workspace_bytes(args, backward=True), q.device)
        st = sla_delta_backward(args, saved, grad_o, _stride(grad_o), grad_last, dq, dk, dv,
                                dbeta, dgate, dstate, work, _raw_stream(q))
        if st != SLA_OK:
            raise SlaError(st, "sla_delta_backward")
        return dq, dk, dv, dbeta, dgate, dstate, None, None


def delta_rule(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
               gate: torch.Tensor, state: Optional[torch.Tensor] = None,
               scale: Optional[float] = None, lengths: Optional[torch.Tensor] = None,
               stream=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """The gated delta rule over whole sequences: (o, last state).

    q, k [batch, tokens, key heads, dk] and v [batch, tokens, value heads, dv]
    of one type (float32, float16, bfloat16; any strides with the last
    dimension contiguous, else they are copied); beta and gate (the log of
    the decay) [batch, tokens, value heads] float32; state [batch, value
    heads, dk, dv] float32, zero by default; scale dk ** -0.5 by default;
    lengths [batch] int32: the tokens of each sequence that are in use (the
    others are not read into any result and answer 0).  Gates are logs of
    decays, 0 or less: where the gates of a run of tokens within a chunk sum to
    more than 2, or one is NaN, the head answers NaN from there on (and may from
    the chunk's first token).  Differentiable in q, k, v, beta, gate and state,
    once, in reverse mode.  Workspaces and outputs come from torch's allocator
    on the stream that the call runs on (``stream``, or the current one)."""
    if torch.is_grad_enabled() or _in_dual_level():
        inputs = q, k, v, beta, gate, state, scale, lengths
        if stream is None:
            return DeltaRule.apply(*inputs)
        with torch.cuda.stream(stream):
            return DeltaRule.apply(*inputs)
    device = _check_rule(q, k, v, beta, gate, state, lengths, 2)
    scale = q.shape[-1] ** -0.5 if scale is None else float(scale)
    with _on(device, stream):
        q, k, v = _rows(q), _rows(k), _rows(v, tokens=True)
        return _forward(q, k, v, beta, gate, state, scale, lengths, False)[:2]


def delta_rule_step(q: torch.Tensor, k: torch.Tensor, v: torch.Tensor, beta: torch.Tensor,
                    gate: torch.Tensor, state: torch.Tensor, scale: Optional[float] = None,
                    slots: Optional[torch.Tensor] = None, out: Optional[torch.Tensor] = None,
                    stream=None) -> torch.Tensor:
    """One token of each sequence: o [batch, value heads, dv], the states
    updated in place.  q, k [batch, key heads, dk], v [batch, value heads,
    dv], beta, gate [batch, value heads]; state [slots, value heads, dk, dv]
    float32, contiguous: a pool, of which sequence b owns state[slots[b]]
    (slots int32, all different; without them state[b]).  A slot outside the
    pool marks a place with no request: its o is 0.  Any gate is taken as the
    formulas stand.  Autograd sees the update as one in place.  It has no derivatives and refuses tensors that ask for them
    (under ``torch.no_grad()`` none does)."""
    device = _check_rule(q, k, v, beta, gate, None, None, 1)
    vs, dk = v.shape, q.shape[-1]
    _need(state.dim() == 4, "state must have 4 dimensions")
    _like(state, "state", (state.shape[0], vs[1], dk, vs[2]), torch.float32, device)
    _need(state.is_contiguous(), "state must be contiguous")
    if slots is not None:
        _like(slots, "slots", (vs[0],), torch.int32, device)
        _need(slots.is_contiguous(), "slots must be contiguous")
    elif state.shape[0] < vs[0]:
        raise ValueError(f"{state.shape[0]} states for {vs[0]} sequences")
    if out is not None:
        _like(out, "out", vs, v.dtype, device)
        _need(vs[2] == 1 or out.stride(-1) == 1, "out's last dimension must be contiguous")
    if _tracked(q, k, v, beta, gate, state, *(() if out is None else (out,))):
        raise ValueError("delta_rule_step has no derivatives: call it under torch.no_grad(), "
                         "or delta_rule on sequences of one token")
    scale = dk ** -0.5 if scale is None else float(scale)
    with _on(device, stream):
        q, k, v = _rows(q), _rows(k), _rows(v)
        o = torch.empty(vs, dtype=v.dtype, device=v.device) if out is None else out
        st = sla_delta_step(_make_args(q, k, v, beta, gate, scale, None, tokens=False), state,
                            slots, o, _stride(o, False), _raw_stream(v))
    if st != SLA_OK:
        raise SlaError(st, "sla_delta_step")
    increment_version((state, o))
    return o
