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
leave_enter_backward).  Forward-mode differentiation is refused
(NotImplementedError).  x and what is shaped like it is fp32 or bf16; y, h
and the gate are of one type, x's or bf16; coefficients and weights are fp32
or bf16 each.  Arithmetic is fp32, every result is rounded once.
"""
from __future__ import annotations

import struct
from collections import namedtuple

import torch
from torch.autograd import forward_ad
from torch.autograd.function import once_differentiable

from . import _DT, _lib
from ._lib import HCB_ACT_LINEAR, HCB_ACT_SIGMOID, HCB_ACT_SILU, HCB_MAX_CHANNELS, HCB_MAX_STREAMS, check

__all__ = ["enter", "enter_backward", "leave", "leave_backward", "leave_enter", "leave_enter_backward",
           "workspace_bytes", "EnterGrads", "LeaveGrads", "LeaveEnterGrads"]

_ACT = {"sigmoid": HCB_ACT_SIGMOID, "silu": HCB_ACT_SILU, "linear": HCB_ACT_LINEAR}

EnterGrads = namedtuple("EnterGrads", "dx da dweight")
LeaveGrads = namedtuple("LeaveGrads", "dx dy dP db dgate dweight")
LeaveEnterGrads = namedtuple("LeaveEnterGrads", "dx dy dP db dgate dweight da_next dweight_next")

# hcb_args packed in one call (a ctypes structure filled field by field takes
# longer than the smallest kernels): T; S C, seven types, act, norm; eps
# eps_next scale; x y gate P a b w w_next dout dh dres out_in; their strides;
# h out dx dy dgate dP da db dw dw_next workspace, workspace_bytes
_ARGS = struct.Struct("<q11i3f12Q14q11QQ")
_MAX_STRIDE = 2 ** 29 - 1
_NONE = (None, 0, 0, 0)  # a tensor that is not there: itself, address, type, stride
_raw_stream = torch._C._cuda_getCurrentRawStream
_functions = {}
_module = None


def _plain():
    """The extension module for plain arguments (contiguous tensors on the
    current device, without tangents): its functions return None where anything else is asked
    or is wrong, and the code here does the call in full."""
    global _module
    if _module is None:
        _module = _lib.binding()
    return _module


def _call(name, dev, args):
    f = _functions.get(name)
    if f is None:
        f = _functions[name] = getattr(_lib.lib(), name)
    if dev == torch.cuda.current_device():
        status = f(args, _raw_stream(dev))
    else:
        with torch.cuda.device(dev):
            status = f(args, _raw_stream(dev))
    if status:
        check(status, name)


def _wrong(t, name, shape, dtype, dev):
    """Say what is wrong with a tensor."""
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if t.dtype not in _DT:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, t.dtype))
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if dev is not None and t.get_device() != dev:
        raise ValueError("%s must be on cuda:%d, got %s" % (name, dev, t.device))
    if shape is not None and t.shape != shape:
        raise ValueError("%s must have shape %s, got %s" % (name, tuple(shape), tuple(t.shape)))
    raise ValueError("%s must be %s, got %s" % (name, dtype, t.dtype))


def _flat(t, inner):
    """t with its leading dimensions as one (a view where their strides allow
    it), the last dimension contiguous.  Rows further apart than the library's
    strides go are copied: they are few (the last tokens of long buffers), or
    would not fit the GPU."""
    if t.dim() != inner + 1:
        t = t.flatten(0, t.dim() - inner - 1) if t.dim() > inner else t.unsqueeze(0)
    if t.shape[-1] > 1 and t.stride(-1) != 1 or max(t.stride()) > _MAX_STRIDE:
        t = t.contiguous()
    return t


def _x(x):
    """(shape, leading shape, T, S, C, device) of the streams."""
    if not isinstance(x, torch.Tensor) or x.dtype not in _DT or not x.is_cuda:
        _wrong(x, "x", None, None, None)
    shape = x.shape
    if len(shape) < 2:
        raise ValueError("x must have shape [..., streams, channels], got %s" % (tuple(shape),))
    S, C = shape[-2], shape[-1]
    if not (1 <= S <= HCB_MAX_STREAMS and 1 <= C <= HCB_MAX_CHANNELS):
        raise ValueError("x must have 1 to %d streams and 1 to %d channels, got %s"
                         % (HCB_MAX_STREAMS, HCB_MAX_CHANNELS, tuple(shape)))
    return shape, shape[:-2], x.numel() // (S * C), S, C, x.get_device()


def _streams(t, name, shape, dtype, dev):
    """(tensor, address, token stride, stream stride) of x or what is shaped like it."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _wrong(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t, t.data_ptr(), shape[-2] * shape[-1], shape[-1]
    t = _flat(t, 2)
    return t, t.data_ptr(), t.stride(0), t.stride(1)


def _row(t, name, shape, dtype, dev):
    """(tensor, address, token stride) of a row of C channels to a token."""
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype != dtype or t.get_device() != dev:
        _wrong(t, name, shape, dtype, dev)
    if t.is_contiguous():
        return t, t.data_ptr(), shape[-1]
    t = _flat(t, 1)
    return t, t.data_ptr(), t.stride(0)


def _few(t, name, shape, inner, dev):
    """(tensor, address, type, token stride) of coefficients, or of a weight (inner 0)."""
    if t is None:
        return _NONE
    if not isinstance(t, torch.Tensor) or t.shape != shape or t.dtype not in _DT or t.get_device() != dev:
        _wrong(t, name, shape, "float32 or bfloat16", dev)
    kind = _DT[t.dtype]
    if t.is_contiguous():
        return t, t.data_ptr(), kind, 0 if inner == 0 else shape[-1] if inner == 1 else shape[-1] * shape[-1]
    if inner == 0:
        t = t.contiguous()
        return t, t.data_ptr(), kind, 0
    t = _flat(t, inner)
    if inner == 2 and t.stride(1) != shape[-1]:
        t = t.contiguous()
    return t, t.data_ptr(), kind, t.stride(0)


def _y_type(dtype, x, name):
    kind = _DT.get(dtype)
    if kind is None:
        raise TypeError("%s must be float32 or bfloat16, got %s" % (name, dtype))
    if kind == 0 and x.dtype == torch.bfloat16:
        raise TypeError("%s must be bfloat16 where x is" % name)
    return kind


def _gate(gate, act, shape, dtype, dev):
    """(act, address, token stride, tensor) of the gate."""
    if gate is None:
        return 0, 0, 0, None
    kind = _ACT.get(act)
    if kind is None:
        raise ValueError("act must be one of %s, got %r" % (", ".join(sorted(_ACT)), act))
    t, ptr, ts = _row(gate, "gate", shape, dtype, dev)
    return kind, ptr, ts, t


def _like(t, wanted=True):
    """A new contiguous tensor for the gradient of t, if it is wanted, and its address."""
    if t is None or not wanted:
        return None, 0
    if not isinstance(t, torch.Tensor):
        raise TypeError("expected a torch.Tensor, got %s" % type(t).__name__)
    g = torch.empty(t.shape, dtype=t.dtype, device=t.device)
    return g, g.data_ptr()


def _scratch(workspace, T, C, weights, device):
    need = workspace_bytes(T, C, weights) if weights else 0
    if need == 0:
        return None, 0, 0
    if workspace is None:
        workspace = torch.empty(need, dtype=torch.uint8, device=device)
    elif workspace.device != device or not workspace.is_contiguous() \
            or workspace.numel() * workspace.element_size() < need:
        raise ValueError("workspace needs %d bytes on %s" % (need, device))
    return workspace, workspace.data_ptr(), need


def workspace_bytes(tokens: int, channels: int, weights: int = 1) -> int:
    """Bytes of scratch of a backward pass with `weights` weight gradients
    (leave_enter_backward: up to 2)."""
    return _lib.lib().hcb_workspace_bytes(tokens, channels, weights)


def _enter(x, a, weight, eps, out_dtype):
    h = _plain().enter(x, a, weight, eps, -1 if out_dtype is None else _DT.get(out_dtype, 2))
    if h is not None:
        return h
    shape, lead, T, S, C, dev = _x(x)
    dtype = out_dtype or x.dtype
    yk = _y_type(dtype, x, "out_dtype")
    x, xp, x_ts, x_ss = _streams(x, "x", shape, x.dtype, dev)
    a, ap, ak, a_ts = _few(a, "a", shape[:-1], 1, dev)
    weight, wp, wk, _ = _few(weight, "weight", shape[-1:], 0, dev)
    h = torch.empty((*lead, C), dtype=dtype, device=x.device)
    _call("hcb_enter", dev, _ARGS.pack(
        T, S, C, _DT[x.dtype], yk, wk, 0, 0, ak, 0, 0, 1, eps, 0.0, 0.0,
        xp, 0, 0, 0, ap, 0, wp, 0, 0, 0, 0, 0,
        x_ts, x_ss, 0, 0, 0, a_ts, 0, 0, 0, 0, 0, 0, 0, 0,
        h.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0, 0))
    return h


_ALL = -1  # every gradient; otherwise bit k stands for the k-th of a function's results


def _enter_backward(dh, x, a, weight, eps, dres, workspace, want):
    if workspace is None:
        got = _plain().enter_backward(dh, x, a, weight, eps, dres, want)
        if got is not None:
            return got
    _no_tangent("enter_backward", dh, x, a, weight, dres)
    shape, lead, T, S, C, dev = _x(x)
    if not isinstance(dh, torch.Tensor):
        _wrong(dh, "dh", None, None, None)
    yk = _y_type(dh.dtype, x, "dh")
    dh, hp, h_ts = _row(dh, "dh", torch.Size((*lead, C)), dh.dtype, dev)
    rp = r_ts = r_ss = 0
    if dres is not None:
        dres, rp, r_ts, r_ss = _streams(dres, "dres", shape, x.dtype, dev)
    dx, dxp = _like(x, want & 1)
    da, dap = _like(a, want & 2)
    dw, dwp = _like(weight, want & 4)
    x, xp, x_ts, x_ss = _streams(x, "x", shape, x.dtype, dev)
    a, ap, ak, a_ts = _few(a, "a", shape[:-1], 1, dev)
    weight, wp, wk, _ = _few(weight, "weight", shape[-1:], 0, dev)
    workspace, wsp, ws = _scratch(workspace, T, C, dw is not None, x.device)
    _call("hcb_enter_backward", dev, _ARGS.pack(
        T, S, C, _DT[x.dtype], yk, wk, 0, 0, ak, 0, 0, 1, eps, 0.0, 0.0,
        xp, 0, 0, 0, ap, 0, wp, 0, 0, hp, rp, 0,
        x_ts, x_ss, 0, 0, 0, a_ts, 0, 0, 0, h_ts, r_ts, r_ss, 0, 0,
        0, 0, dxp, 0, 0, 0, dap, 0, dwp, 0, wsp, ws))
    return dx, da, dw


def enter_backward(dh: torch.Tensor, x: torch.Tensor, a: torch.Tensor = None, weight: torch.Tensor = None, *,
                   eps: float = 1e-6, dres: torch.Tensor = None, workspace: torch.Tensor = None) -> EnterGrads:
    """The gradients of enter: (dx, da, dweight), da and dweight None where
    a and weight are.  dres, shaped like x, is added to dx: the gradient that
    the streams have from elsewhere.  workspace: a uint8 tensor of
    workspace_bytes (allocated here if not given)."""
    return EnterGrads._make(_enter_backward(dh, x, a, weight, eps, dres, workspace, _ALL))


def _leave(x, y, P, b, gate, act, weight, norm, scale, eps, want_h, a_next, weight_next, eps_next):
    got = _plain().leave(x, y, P, b, gate, _ACT.get(act, -1), weight, norm, scale, eps, want_h, a_next, weight_next,
                         eps_next)
    if got is not None:
        return got
    shape, lead, T, S, C, dev = _x(x)
    if not isinstance(y, torch.Tensor):
        _wrong(y, "y", None, None, None)
    yt, row = y.dtype, torch.Size((*lead, C))
    yk = _y_type(yt, x, "y")
    y, yp, y_ts = _row(y, "y", row, yt, dev)
    act, gp, g_ts, gate = _gate(gate, act, row, yt, dev)
    x, xp, x_ts, x_ss = _streams(x, "x", shape, x.dtype, dev)
    P, Pp, pk, P_ts = _few(P, "P", (*lead, S, S), 2, dev)
    b, bp, bk, b_ts = _few(b, "b", shape[:-1], 1, dev)
    weight, wp, wk, _ = _few(weight, "weight", shape[-1:], 0, dev)
    out = torch.empty(shape, dtype=x.dtype, device=x.device)
    h, hp = None, 0
    ap = ak = a_ts = wnp = wnk = 0
    if want_h:
        a_next, ap, ak, a_ts = _few(a_next, "a_next", shape[:-1], 1, dev)
        weight_next, wnp, wnk, _ = _few(weight_next, "weight_next", shape[-1:], 0, dev)
        h = torch.empty(row, dtype=yt, device=x.device)
        hp = h.data_ptr()
    _call("hcb_leave", dev, _ARGS.pack(
        T, S, C, _DT[x.dtype], yk, wk, wnk, pk, ak, bk, act, bool(norm), eps, eps_next, scale,
        xp, yp, gp, Pp, ap, bp, wp, wnp, 0, 0, 0, 0,
        x_ts, x_ss, y_ts, g_ts, P_ts, a_ts, b_ts, 0, 0, 0, 0, 0, 0, 0,
        hp, out.data_ptr(), 0, 0, 0, 0, 0, 0, 0, 0, 0, 0))
    return out, h


def _leave_backward(dout, dh, out, x, y, P, b, gate, act, weight, norm, scale, eps, a_next, weight_next, eps_next,
                    workspace, want=_ALL):
    if workspace is None:
        got = _plain().leave_backward(x, y, P, b, gate, _ACT.get(act, -1), weight, norm, scale, eps, dout, dh, out,
                                      a_next, weight_next, eps_next, want)
        if got is not None:
            return got
    _no_tangent("leave_backward" if dh is None else "leave_enter_backward", dout, dh, out, x, y, P, b, gate, weight, a_next,
                weight_next)
    shape, lead, T, S, C, dev = _x(x)
    if not isinstance(y, torch.Tensor):
        _wrong(y, "y", None, None, None)
    xt, yt, row = x.dtype, y.dtype, torch.Size((*lead, C))
    yk = _y_type(yt, x, "y")
    # without a mixing matrix dx is dout, unless h's gradient is added to it
    dx, dxp = _like(x, want & 1 or dh is not None) if P is not None or dh is not None else (dout, 0)
    dy, dyp = _like(y, want & 2)
    dP, dPp = _like(P, want & 4)
    db, dbp = _like(b, want & 8)
    dgate, dgp = _like(gate, want & 16)
    dw, dwp = _like(weight, want & 32)
    dout, dop, do_ts, do_ss = _streams(dout, "dout", shape, xt, dev)
    y, yp, y_ts = _row(y, "y", row, yt, dev)
    act, gp, g_ts, gate = _gate(gate, act, row, yt, dev)
    P, Pp, pk, P_ts = _few(P, "P", (*lead, S, S), 2, dev)
    b, bp, bk, b_ts = _few(b, "b", shape[:-1], 1, dev)
    weight, wp, wk, _ = _few(weight, "weight", shape[-1:], 0, dev)
    xp = x_ts = x_ss = 0
    if P is not None:
        x, xp, x_ts, x_ss = _streams(x, "x", shape, xt, dev)
    da = dwn = None
    hp = h_ts = op = o_ts = o_ss = ap = ak = a_ts = wnp = wnk = dap = dwnp = 0
    if dh is not None:
        dh, hp, h_ts = _row(dh, "dh", row, yt, dev)
        out, op, o_ts, o_ss = _streams(out, "out", shape, xt, dev)
        da, dap = _like(a_next, want & 64)
        dwn, dwnp = _like(weight_next, want & 128)
        a_next, ap, ak, a_ts = _few(a_next, "a_next", shape[:-1], 1, dev)
        weight_next, wnp, wnk, _ = _few(weight_next, "weight_next", shape[-1:], 0, dev)
    workspace, wsp, ws = _scratch(workspace, T, C, (dw is not None) + (dwn is not None), x.device)
    _call("hcb_leave_backward", dev, _ARGS.pack(
        T, S, C, _DT[xt], yk, wk, wnk, pk, ak, bk, act, bool(norm), eps, eps_next, scale,
        xp, yp, gp, Pp, ap, bp, wp, wnp, dop, hp, 0, op,
        x_ts, x_ss, y_ts, g_ts, P_ts, a_ts, b_ts, do_ts, do_ss, h_ts, 0, 0, o_ts, o_ss,
        0, 0, dxp, dyp, dgp, dPp, dap, dbp, dwp, dwnp, wsp, ws))
    return dx, dy, dP, db, dgate, dw, da, dwn


def leave_backward(dout: torch.Tensor, x: torch.Tensor, y: torch.Tensor, P: torch.Tensor = None,
                   b: torch.Tensor = None, *, gate: torch.Tensor = None, act: str = "sigmoid",
                   weight: torch.Tensor = None, norm: bool = True, scale: float = 1.0, eps: float = 1e-6,
                   workspace: torch.Tensor = None) -> LeaveGrads:
    """The gradients of leave: (dx, dy, dP, db, dgate, dweight), None where
    the tensor is.  Without P, dx is dout itself."""
    return LeaveGrads._make(_leave_backward(dout, None, None, x, y, P, b, gate, act, weight, norm, scale, eps, None, None,
                                            0.0, workspace)[:6])


def leave_enter_backward(dout: torch.Tensor, dh: torch.Tensor, out: torch.Tensor, x: torch.Tensor, y: torch.Tensor,
                         P: torch.Tensor = None, b: torch.Tensor = None, *, gate: torch.Tensor = None,
                         act: str = "sigmoid", weight: torch.Tensor = None, norm: bool = True, scale: float = 1.0,
                         eps: float = 1e-6, a_next: torch.Tensor = None, weight_next: torch.Tensor = None,
                         eps_next: float = 1e-6, workspace: torch.Tensor = None) -> LeaveEnterGrads:
    """The gradients of leave_enter, from those of both its results and its
    stored result `out`, in one pass: (dx, dy, dP, db, dgate, dweight,
    da_next, dweight_next), None where the tensor is."""
    return LeaveEnterGrads._make(_leave_backward(dout, dh, out, x, y, P, b, gate, act, weight, norm, scale, eps, a_next,
                                                 weight_next, eps_next, workspace))


def _bits(needed):
    """Which gradients autograd asks for, as `want` has them."""
    return sum(1 << k for k, n in enumerate(needed) if n)


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
        return (*_enter_backward(dh, x, a, weight, ctx.eps, None, None, _bits(ctx.needs_input_grad)), None, None)


class _Leave(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, P, b, gate, weight, *how):
        ctx.save_for_backward(None if P is None else x, y, P, b, gate, weight)
        ctx.how = how
        act, norm, scale, eps = how
        return _leave(x, y, P, b, gate, act, weight, norm, scale, eps, False, None, None, 0.0)[0]

    @staticmethod
    @once_differentiable
    def backward(ctx, dout):
        x, y, P, b, gate, weight = ctx.saved_tensors
        act, norm, scale, eps = ctx.how
        g = _leave_backward(dout, None, None, dout if x is None else x, y, P, b, gate, act, weight, norm, scale, eps, None, None,
                            0.0, None, _bits(ctx.needs_input_grad))
        return (*g[:6], None, None, None, None)


class _LeaveEnter(torch.autograd.Function):
    @staticmethod
    def forward(ctx, x, y, P, b, gate, weight, a_next, weight_next, *how):
        act, norm, scale, eps, eps_next = how
        out, h = _leave(x, y, P, b, gate, act, weight, norm, scale, eps, True, a_next, weight_next, eps_next)
        # without a mixing matrix the gradients do not need x's values
        ctx.save_for_backward(None if P is None else x, y, P, b, gate, weight, a_next, weight_next, out)
        ctx.how = how
        ctx.set_materialize_grads(False)
        return out, h

    @staticmethod
    @once_differentiable
    def backward(ctx, dout, dh):
        x, y, P, b, gate, weight, a_next, weight_next, out = ctx.saved_tensors
        act, norm, scale, eps, eps_next = ctx.how
        # results that the loss does not have: without h's gradient it is leave's,
        # and a zero for that of the streams is one row, repeated
        if dout is None and dh is None:
            return (None,) * 13
        if dout is None:
            dout = torch.zeros(out.shape[-1], dtype=out.dtype, device=out.device).expand(out.shape)
        g = _leave_backward(dout, dh, out, out if x is None else x, y, P, b, gate, act, weight, norm, scale, eps, a_next,
                            weight_next, eps_next, None, _bits(ctx.needs_input_grad))
        return (*g, None, None, None, None, None)


def _tangent(tensors):
    """Whether one of them carries a forward-mode tangent."""
    return forward_ad._current_level >= 0 and any(
        isinstance(t, torch.Tensor) and forward_ad.unpack_dual(t).tangent is not None for t in tensors)


def _no_tangent(name, *tensors):
    if _tangent(tensors):
        raise NotImplementedError("%s has no forward-mode derivative" % name)


def _learns(*tensors):
    """Whether the call goes through its autograd function: to record it, or
    to have a tangent refused (which grad mode has no say in)."""
    if _tangent(tensors):
        return True
    if not torch.is_grad_enabled():
        return False
    for t in tensors:
        if t is not None and getattr(t, "requires_grad", False):
            return True
    return False


def enter(x: torch.Tensor, a: torch.Tensor = None, weight: torch.Tensor = None, *, eps: float = 1e-6,
          out_dtype=None) -> torch.Tensor:
    """A block's input from the residual streams x [..., S, C]:
    u = sum_s a_s x_s, h = weight * u / sqrt(mean u^2 + eps), [..., C].

    a [..., S]: the read coefficients (ones if None); weight [C] (ones if
    None); out_dtype: h's type (x's if None; x fp32 may give bf16)."""
    h = _plain().enter(x, a, weight, eps, -1 if out_dtype is None else _DT.get(out_dtype, 2))
    if h is not None:
        return h
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
    got = _plain().leave(x, y, P, b, gate, _ACT.get(act, -1), weight, norm, scale, eps, False, None, None, 0.0)
    if got is not None:
        return got[0]
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
    got = _plain().leave(x, y, P, b, gate, _ACT.get(act, -1), weight, norm, scale, eps, True, a_next, weight_next,
                         eps_next)
    if got is not None:
        return got
    if _learns(x, y, P, b, gate, weight, a_next, weight_next):
        return _LeaveEnter.apply(x, y, P, b, gate, weight, a_next, weight_next, act, norm, scale, eps, eps_next)
    return _leave(x, y, P, b, gate, act, weight, norm, scale, eps, True, a_next, weight_next, eps_next)
