"""The operators around one block of a network with hyper-connections:
Python binding of include/hc_block.h.  Argument marshalling only; every step
runs in the library's kernels.

The residual is S streams of C channels per token, x [..., S, C].

    h = enter(x, a, weight)                       # u = sum_s a_s x_s, RMS-normalised
    y = block(h)
    x = leave(x, y, project(logits), b, weight=w_post, gate=g, act="sigmoid")
    x, h = leave_enter(x, y, P, b, a_next=a2, weight_next=w2)   # and the next block's input

All three are differentiable in every tensor they take.  The gradients are
also there as functions of their own (enter_backward, leave_backward,
leave_enter_backward).  x and what is shaped like it is fp32 or bf16; y, h
and the gate are of one type, x's or bf16; coefficients and weights are fp32
or bf16 each.  Arithmetic is fp32, every result is rounded once.
"""
from __future__ import annotations

import ctypes
from collections import namedtuple

import torch
from torch.autograd.function import once_differentiable

from . import _DT, _on_device, _ptr, _stream
from ._lib import (HCB_ACT_LINEAR, HCB_ACT_NONE, HCB_ACT_SIGMOID, HCB_ACT_SILU, HCB_MAX_CHANNELS, HCB_MAX_STREAMS,
                   HcbArgs, check, lib)

__all__ = ["enter", "enter_backward", "leave", "leave_backward", "leave_enter", "leave_enter_backward",
           "EnterGrads", "LeaveGrads", "LeaveEnterGrads"]

_ACT = {"sigmoid": HCB_ACT_SIGMOID, "silu": HCB_ACT_SILU, "linear": HCB_ACT_LINEAR}

EnterGrads = namedtuple("EnterGrads", "dx da dweight")
LeaveGrads = namedtuple("LeaveGrads", "dx dy dP db dgate dweight")
LeaveEnterGrads = namedtuple("LeaveEnterGrads", "dx dy dP db dgate dweight da_next dweight_next")


def _need(t, name, like=None):
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in _DT:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if like is not None and t.device != like.device:
        raise ValueError("%s must be on %s, got %s" % (name, like.device, t.device))


def _flat(t, inner):
    """t with its leading dimensions as one (a view where their strides allow
    it), the last dimension contiguous."""
    if t.dim() != inner + 1:
        t = t.flatten(0, t.dim() - inner - 1) if t.dim() > inner else t.unsqueeze(0)
    if t.stride(-1) != 1 and t.shape[-1] > 1:
        t = t.contiguous()
    return t


class _Call:
    """The arguments of one call: an hcb_args, and the tensors it points to."""

    def __init__(self, x):
        _need(x, "x")
        if x.dim() < 2:
            raise ValueError("x must have shape [..., streams, channels], got %s" % (tuple(x.shape),))
        self.lead, (self.S, self.C) = x.shape[:-2], x.shape[-2:]
        if not (1 <= self.S <= HCB_MAX_STREAMS and 1 <= self.C <= HCB_MAX_CHANNELS):
            raise ValueError("x must have 1 to %d streams and 1 to %d channels, got %s"
                             % (HCB_MAX_STREAMS, HCB_MAX_CHANNELS, tuple(x.shape)))
        self.x, self.device, self.keep = x, x.device, []
        self.T = x.numel() // (self.S * self.C)
        self.args = HcbArgs(T=self.T, S=self.S, C=self.C, x_dtype=_DT[x.dtype], norm=1)

    def streams(self, t, name, field, ts, ss):
        if t is not self.x:
            _need(t, name, self.x)
            if t.shape != self.x.shape or t.dtype != self.x.dtype:
                raise ValueError("%s must have x's shape and dtype" % name)
        t = _flat(t, 2)
        self.keep.append(t)
        a = self.args
        setattr(a, field, t.data_ptr())
        setattr(a, ts, t.stride(0))
        setattr(a, ss, t.stride(1))

    def row(self, t, name, field, ts, dtype=None):
        """A row of C channels per token, of y's type."""
        _need(t, name, self.x)
        if t.shape[:-1] != self.lead or t.shape[-1] != self.C:
            raise ValueError("%s must have shape %s, got %s" % (name, (*self.lead, self.C), tuple(t.shape)))
        if dtype is not None and t.dtype != dtype:
            raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))
        t = _flat(t, 1)
        self.keep.append(t)
        setattr(self.args, field, t.data_ptr())
        setattr(self.args, ts, t.stride(0))

    def y_type(self, dtype, name):
        if dtype not in _DT:
            raise TypeError("%s must be float32 or bfloat16, got %s" % (name, dtype))
        if dtype == torch.float32 and self.x.dtype == torch.bfloat16:
            raise TypeError("%s must be bfloat16 where x is" % name)
        self.args.y_dtype = _DT[dtype]

    def coefficients(self, t, name, field, kind, ts, shape):
        if t is None:
            return
        _need(t, name, self.x)
        if t.shape != (*self.lead, *shape):
            raise ValueError("%s must have shape %s, got %s" % (name, (*self.lead, *shape), tuple(t.shape)))
        t = _flat(t, len(shape))
        if len(shape) == 2 and t.stride(1) != shape[1]:
            t = t.contiguous()
        self.keep.append(t)
        setattr(self.args, field, t.data_ptr())
        setattr(self.args, kind, _DT[t.dtype])
        setattr(self.args, ts, t.stride(0))

    def weight(self, t, name, field, kind):
        if t is None:
            return
        _need(t, name, self.x)
        if t.shape != (self.C,):
            raise ValueError("%s must have shape (%d,), got %s" % (name, self.C, tuple(t.shape)))
        t = t.contiguous()
        self.keep.append(t)
        setattr(self.args, field, t.data_ptr())
        setattr(self.args, kind, _DT[t.dtype])

    def new(self, field, shape, dtype):
        t = torch.empty(shape, dtype=dtype, device=self.device)
        setattr(self.args, field, t.data_ptr())
        return t

    def like(self, field, t):
        """A new tensor for the gradient of t (None where t is)."""
        return None if t is None else self.new(field, t.shape, t.dtype)

    def gated(self, gate, act, y):
        if gate is None:
            return
        if act not in _ACT:
            raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(_ACT)), act))
        self.args.act = _ACT[act]
        self.row(gate, "gate", "gate", "gate_ts", y.dtype)

    def scratch(self, workspace, weights):
        need = lib().hcb_workspace_bytes(self.T, self.C, weights)
        if need == 0:
            return
        if workspace is None:
            workspace = torch.empty(need, dtype=torch.uint8, device=self.device)
        elif workspace.device != self.device or not workspace.is_contiguous() \
                or workspace.numel() * workspace.element_size() < need:
            raise ValueError("workspace needs %d bytes on %s" % (need, self.device))
        self.keep.append(workspace)
        self.args.workspace = workspace.data_ptr()
        self.args.workspace_bytes = need

    def run(self, name):
        with _on_device(self.x):
            check(getattr(lib(), name)(ctypes.byref(self.args), _stream(self.x)), name)


def workspace_bytes(tokens: int, channels: int, weights: int = 1) -> int:
    """Bytes of scratch of a backward pass with `weights` weight gradients
    (leave_enter_backward: up to 2)."""
    return lib().hcb_workspace_bytes(tokens, channels, weights)


def _enter(x, a, weight, eps, out_dtype):
    c = _Call(x)
    dtype = out_dtype or x.dtype
    c.y_type(dtype, "out_dtype")
    c.args.eps = eps
    c.streams(x, "x", "x", "x_ts", "x_ss")
    c.coefficients(a, "a", "a", "a_dtype", "a_ts", (c.S,))
    c.weight(weight, "weight", "w", "w_dtype")
    h = c.new("h", (*c.lead, c.C), dtype)
    c.run("hcb_enter")
    return h


def enter_backward(dh: torch.Tensor, x: torch.Tensor, a: torch.Tensor = None, weight: torch.Tensor = None, *,
                   eps: float = 1e-6, dres: torch.Tensor = None, workspace: torch.Tensor = None) -> EnterGrads:
    """The gradients of enter: (dx, da, dweight), da and dweight None where
    a and weight are.  dres, shaped like x, is added to dx: the gradient that
    the streams have from elsewhere.  workspace: a uint8 tensor of
    workspace_bytes (allocated here if not given)."""
    c = _Call(x)
    _need(dh, "dh", x)
    c.y_type(dh.dtype, "dh")
    c.args.eps = eps
    c.streams(x, "x", "x", "x_ts", "x_ss")
    c.row(dh, "dh", "dh", "dh_ts")
    c.coefficients(a, "a", "a", "a_dtype", "a_ts", (c.S,))
    c.weight(weight, "weight", "w", "w_dtype")
    if dres is not None:
        c.streams(dres, "dres", "dres", "dres_ts", "dres_ss")
    got = EnterGrads(c.like("dx", x), c.like("da", a), c.like("dw", weight))
    if weight is not None:
        c.scratch(workspace, 1)
    c.run("hcb_enter_backward")
    return got


def _leave_inputs(c, x, y, P, b, gate, act, weight, norm, scale, eps):
    _need(y, "y", x)
    c.y_type(y.dtype, "y")
    c.args.norm, c.args.scale, c.args.eps = bool(norm), scale, eps
    c.row(y, "y", "y", "y_ts")
    c.gated(gate, act, y)
    c.coefficients(P, "P", "P", "p_dtype", "P_ts", (c.S, c.S))
    c.coefficients(b, "b", "b", "b_dtype", "b_ts", (c.S,))
    c.weight(weight, "weight", "w", "w_dtype")


def _leave(x, y, P, b, gate, act, weight, norm, scale, eps, want_h, a_next, weight_next, eps_next):
    c = _Call(x)
    _leave_inputs(c, x, y, P, b, gate, act, weight, norm, scale, eps)
    c.streams(x, "x", "x", "x_ts", "x_ss")
    out = c.new("out", x.shape, x.dtype)
    h = None
    if want_h:
        c.args.eps_next = eps_next
        c.coefficients(a_next, "a_next", "a", "a_dtype", "a_ts", (c.S,))
        c.weight(weight_next, "weight_next", "w_next", "wn_dtype")
        h = c.new("h", (*c.lead, c.C), y.dtype)
    c.run("hcb_leave")
    return out, h


def _leave_backward(dout, dh, out, x, y, P, b, gate, act, weight, norm, scale, eps, a_next, weight_next, eps_next,
                    workspace):
    c = _Call(x)
    _leave_inputs(c, x, y, P, b, gate, act, weight, norm, scale, eps)
    c.streams(dout, "dout", "dout", "dout_ts", "dout_ss")
    if P is not None:
        c.streams(x, "x", "x", "x_ts", "x_ss")
    # without a mixing matrix dx is dout, unless h's gradient is added to it
    dx = c.new("dx", x.shape, x.dtype) if P is not None or dh is not None else dout
    da = dwn = None
    if dh is not None:
        c.args.eps_next = eps_next
        c.row(dh, "dh", "dh", "dh_ts", y.dtype)
        c.streams(out, "out", "out_in", "out_ts", "out_ss")
        c.coefficients(a_next, "a_next", "a", "a_dtype", "a_ts", (c.S,))
        c.weight(weight_next, "weight_next", "w_next", "wn_dtype")
        da, dwn = c.like("da", a_next), c.like("dw_next", weight_next)
    got = (dx, c.like("dy", y), c.like("dP", P), c.like("db", b), c.like("dgate", gate), c.like("dw", weight))
    c.scratch(workspace, (weight is not None) + (dwn is not None))
    c.run("hcb_leave_backward")
    return got, da, dwn


def leave_backward(dout: torch.Tensor, x: torch.Tensor, y: torch.Tensor, P: torch.Tensor = None,
                   b: torch.Tensor = None, *, gate: torch.Tensor = None, act: str = "sigmoid",
                   weight: torch.Tensor = None, norm: bool = True, scale: float = 1.0, eps: float = 1e-6,
                   workspace: torch.Tensor = None) -> LeaveGrads:
    """The gradients of leave: (dx, dy, dP, db, dgate, dweight), None where
    the tensor is.  Without P, dx is dout itself."""
    return LeaveGrads(*_leave_backward(dout, None, None, x, y, P, b, gate, act, weight, norm, scale, eps, None, None,
                                       0.0, workspace)[0])


def leave_enter_backward(dout: torch.Tensor, dh: torch.Tensor, out: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                         P: torch.Tensor = None, b: torch.Tensor = None, *, gate: torch.Tensor = None,
                         act: str = "sigmoid", weight: torch.Tensor = None, norm: bool = True, scale: float = 1.0,
                         eps: float = 1e-6, a_next: torch.Tensor = None, weight_next: torch.Tensor = None,
                         eps_next: float = 1e-6, workspace: torch.Tensor = None) -> LeaveEnterGrads:
    """The gradients of leave_enter, from those of both its results and its
    stored result `out`, in one pass: (dx, dy, dP, db, dgate, dweight,
    da_next, dweight_next), None where the tensor is."""
    got, da, dwn = _leave_backward(dout, dh, out, x, y, P, b, gate, act, weight, norm, scale, eps, a_next, weight_next,
                                   eps_next, workspace)
    return LeaveEnterGrads(*got, da, dwn)


class _Enter(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, a, weight, eps, out_dtype):
        ctx.save_for_backward(x, a, weight)
        ctx.eps = eps
        return _enter(x, a, weight, eps, out_dtype)

    @staticmethod
    @once_differentiable
    def backward(ctx, dh):
        x, a, weight = ctx.saved_tensors
        return (*enter_backward(dh, x, a, weight, eps=ctx.eps), None, None)


class _Leave(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, P, b, gate, weight, *how):
        ctx.save_for_backward(x, y, P, b, gate, weight)
        ctx.how = how
        act, norm, scale, eps = how
        return _leave(x, y, P, b, gate, act, weight, norm, scale, eps, False, None, None, 0.0)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x, y, P, b, gate, weight = ctx.saved_tensors
        act, norm, scale, eps = ctx.how
        g = leave_backward(dout, x, y, P, b, gate=gate, act=act, weight=weight, norm=norm, scale=scale, eps=eps)
        return (g.dx, g.dy, g.dP, g.db, g.dgate, g.dweight, None, None, None, None)


class _LeaveEnter(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, P, b, gate, weight, a_next, weight_next, *how):
        act, norm, scale, eps, eps_next = how
        out, h = _leave(x, y, P, b, gate, act, weight, norm, scale, eps, True, a_next, weight_next, eps_next)
        ctx.save_for_backward(x, y, P, b, gate, weight, a_next, weight_next, out)
        ctx.how = how
        return out, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dh):
        x, y, P, b, gate, weight, a_next, weight_next, out = ctx.saved_tensors
        act, norm, scale, eps, eps_next = ctx.how
        g = leave_enter_backward(dout, dh, out, x, y, P, b, gate=gate, act=act, weight=weight, norm=norm, scale=scale,
                                 eps=eps, a_next=a_next, weight_next=weight_next, eps_next=eps_next)
        return (g.dx, g.dy, g.dP, g.db, g.dgate, g.dweight, g.da_next, g.dweight_next, None, None, None, None, None)


def _learns(*tensors):
    return torch.is_grad_enabled() and any(isinstance(t, torch.Tensor) and t.requires_grad for t in tensors)


def enter(x: torch.Tensor, a: torch.Tensor = None, weight: torch.Tensor = None, *, eps: float = 1e-6,
          out_dtype=None) -> torch.Tensor:
    """A block's input from the residual streams x [..., S, C]:
    u = sum_s a_s x_s, h = weight * u / sqrt(mean u^2 + eps), [..., C].

    a [..., S]: the read coefficients (ones if None); weight [C] (ones if
    None); out_dtype: h's type (x's if None; x fp32 may give bf16)."""
    if _learns(x, a, weight):
        return _Enter.apply(x, a, weight, eps, out_dtype)
    return _enter(x, a, weight, eps, out_dtype)


def leave(x: torch.Tensor, y: torch.Tensor, P: torch.Tensor = None, b: torch.Tensor = None, *,
          gate: torch.Tensor = None, act: str = "sigmoid", weight: torch.Tensor = None, norm: bool = True,
          scale: float = 1.0, eps: float = 1e-6) -> torch.Tensor:
    """A block's output y [..., C] written back into the streams x [..., S, C]:
    z = weight * y / sqrt(mean y^2 + eps) (weight * y if not norm),
    v = scale * act(gate) * z, x'_i = sum_j P_ij x_j + b_i v.

    P [..., S, S]: the mixing matrices, as project returns them (identity if
    None); b [..., S]: the write coefficients (ones if None); gate [..., C]
    of y's type with act "sigmoid", "silu" or "linear" (no gate if None);
    weight [C] (ones if None)."""
    if _learns(x, y, P, b, gate, weight):
        return _Leave.apply(x, y, P, b, gate, weight, act, norm, scale, eps)
    return _leave(x, y, P, b, gate, act, weight, norm, scale, eps, False, None, None, 0.0)[0]


def leave_enter(x: torch.Tensor, y: torch.Tensor, P: torch.Tensor = None, b: torch.Tensor = None, *,
                gate: torch.Tensor = None, act: str = "sigmoid", weight: torch.Tensor = None, norm: bool = True,
                scale: float = 1.0, eps: float = 1e-6, a_next: torch.Tensor = None,
                weight_next: torch.Tensor = None, eps_next: float = 1e-6):
    """leave, and the next block's input from its result in the same pass:
    returns (x', h) with x' = leave(...) and
    h = enter(x', a_next, weight_next, eps=eps_next), of y's type.

    For a residual of one stream: x' = x + scale * act(gate) * norm(y), and
    the norm of x'."""
    if _learns(x, y, P, b, gate, weight, a_next, weight_next):
        return _LeaveEnter.apply(x, y, P, b, gate, weight, a_next, weight_next, act, norm, scale, eps, eps_next)
    return _leave(x, y, P, b, gate, act, weight, norm, scale, eps, True, a_next, weight_next, eps_next)
