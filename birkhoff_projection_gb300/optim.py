"""AdamW over many tensors in one launch, with moments in 32 or in 8 bits:
Python binding of include/adamw.h.

    opt = AdamW(model.parameters(), lr=1e-3, weight_decay=0.1, state_bits=8, master_weights=True)
    loss.backward()
    opt.step()

The moments (and the fp32 master weights of bf16 parameters) of all
parameters of one type are views of a few packed buffers, in which every
tensor begins on a multiple of 128 elements.  8-bit moments are e4m3 numbers
with one fp32 scale to 128 elements; the second moment is held as its root.
"""
from __future__ import annotations

import struct
from array import array

import torch

from . import _DT
from ._lib import ADAMW_BLOCK, check, lib

__all__ = ["AdamW"]

# adamw_tensor is eight 8-byte fields: p g m v m_scale v_scale master n
_FIELDS = 8
# adamw_opts: p_dtype g_dtype state_bits; lr beta1 beta2 eps weight_decay; step, grad_scale
_OPTS = struct.Struct("<3i4x5dqQ")


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay, one launch for up to 256 tensors of
    a group.

    params: fp32 or bf16 CUDA parameters, contiguous, on one device; a group
    may set its own lr, betas, eps and weight_decay.  state_bits: 32 or 8.
    master_weights: keep an fp32 copy of bf16 parameters and step on that.
    step(grad_scale=t) multiplies every gradient by the fp32 device scalar t.
    A parameter without a gradient is left alone, and so are its moments; all
    parameters share one count of steps (the attribute `steps`)."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2, *,
                 state_bits: int = 32, master_weights: bool = False):
        for name, v in (("lr", lr), ("eps", eps), ("weight_decay", weight_decay)):
            if not 0.0 <= v < float("inf"):
                raise ValueError("%s must be finite and not negative, got %r" % (name, v))
        if len(betas) != 2 or not all(0.0 <= b < 1.0 for b in betas):
            raise ValueError("betas must be two numbers in [0, 1), got %r" % (betas,))
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        self.steps = 0
        self.state_bits, self.master_weights = state_bits, bool(master_weights)
        self._packed, self._ready = None, False
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay))
        self._ready = True
        self._pack()

    def add_param_group(self, group):
        if self._ready:
            raise ValueError("all parameters are given at construction: their state is packed")
        super().add_param_group(group)

    def _pack(self):
        """Allocate the packed state and each parameter's views of it."""
        every = [p for g in self.param_groups for p in g["params"]]
        device = every[0].device
        if device.type != "cuda":
            raise ValueError("parameters must be on one CUDA device")
        for p in every:
            if p.dtype not in _DT:
                raise TypeError("parameters must be float32 or bfloat16, got %s" % p.dtype)
            if not p.is_cuda or p.device != device:
                raise ValueError("parameters must be on one CUDA device")
            if not p.is_contiguous():
                raise ValueError("parameters must be contiguous")
        master = self.master_weights
        if master and any(p.dtype != torch.bfloat16 for p in every):
            raise ValueError("master_weights is for bfloat16 parameters")
        total = sum(-(-p.numel() // ADAMW_BLOCK) for p in every) * ADAMW_BLOCK
        eight = self.state_bits == 8

        def zeros(n, dtype):
            return torch.zeros(n, dtype=dtype, device=device)

        kind = torch.float8_e4m3fn if eight else torch.float32
        second = "exp_avg_sq_root" if eight else "exp_avg_sq"
        self._packed = {"exp_avg": zeros(total, kind), second: zeros(total, kind)}
        if eight:
            for name in ("exp_avg_scale", "exp_avg_sq_root_scale"):
                self._packed[name] = zeros(total // ADAMW_BLOCK, torch.float32)
        if master:
            self._packed["master"] = zeros(total, torch.float32)
        self._device, self._second = device, second
        at = 0
        for p in every:
            n = p.numel()
            state = {}
            for name, buf in self._packed.items():
                if name.endswith("_scale"):
                    state[name] = buf[at // ADAMW_BLOCK:at // ADAMW_BLOCK + -(-n // ADAMW_BLOCK)]
                else:
                    state[name] = buf[at:at + n].view(p.shape)
            if master:
                state["master"].copy_(p.detach())
            self.state[p] = state
            at += -(-n // ADAMW_BLOCK) * ADAMW_BLOCK
        self._tables()

    def _tables(self):
        """Per group and type, the library's table of tensors with the state's addresses filled in."""
        self._plans = []
        for group in self.param_groups:
            for dtype in _DT:
                params = [p for p in group["params"] if p.dtype == dtype and p.numel() > 0]
                if not params:
                    continue
                rows = array("Q")
                for p in params:
                    s = self.state[p]
                    eight, master = self.state_bits == 8, self.master_weights
                    rows.extend((0, 0, s["exp_avg"].data_ptr(), s[self._second].data_ptr(),
                                 s["exp_avg_scale"].data_ptr() if eight else 0,
                                 s["exp_avg_sq_root_scale"].data_ptr() if eight else 0,
                                 s["master"].data_ptr() if master else 0, p.numel()))
                self._plans.append((group, dtype, params, rows))

    def packed(self) -> dict:
        """The packed state buffers: exp_avg and exp_avg_sq (32 bits), or
        exp_avg and exp_avg_sq_root as e4m3 with exp_avg_scale and
        exp_avg_sq_root_scale (8 bits); master with master weights.  The
        tensors follow each other in the order of the parameters, each on a
        multiple of 128 elements."""
        return dict(self._packed)

    @torch.no_grad()
    def step(self, closure=None, *, grad_scale: torch.Tensor = None):
        """One step on the parameters' gradients (fp32 or bf16, contiguous)."""
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1
                                       or grad_scale.device != self._device):
            raise ValueError("grad_scale must be one float32 on %s" % self._device)
        dev = self._device.index
        calls = []  # the tables, and whatever they point to that is not kept elsewhere
        for group, dtype, params, rows in self._plans:
            grads = [p.grad for p in params]
            if any([g is None for g in grads]):  # (`in` would compare tensors)
                some = [k for k, g in enumerate(grads) if g is not None]
                params, grads = [params[k] for k in some], [grads[k] for k in some]
                rows = array("Q", [v for k in some for v in rows[k * _FIELDS:(k + 1) * _FIELDS]])
                if not some:
                    continue
            kinds = {g.dtype for g in grads}
            if not kinds <= _DT.keys() or {g.get_device() for g in grads} != {dev} \
                    or {g.layout for g in grads} != {torch.strided}:
                raise ValueError("gradients must be dense float32 or bfloat16 tensors on %s" % self._device)
            if not all([g.is_contiguous() for g in grads]):
                grads = [g.contiguous() for g in grads]
            table = rows[:]
            view = memoryview(table)
            view[0::_FIELDS] = memoryview(array("Q", [p.data_ptr() for p in params]))
            view[1::_FIELDS] = memoryview(array("Q", [g.data_ptr() for g in grads]))
            for kind in kinds:
                if len(kinds) > 1:
                    mine = array("Q", [v for k, g in enumerate(grads) if g.dtype == kind
                                       for v in table[k * _FIELDS:(k + 1) * _FIELDS]])
                else:
                    mine = table
                calls.append((group, dtype, kind, mine, grads))
        self.steps += 1
        scale = 0 if grad_scale is None else grad_scale.data_ptr()
        f = lib().adamw_step
        with torch.cuda.device(self._device):
            stream = torch._C._cuda_getCurrentRawStream(dev)
            for group, dtype, kind, table, _ in calls:
                beta1, beta2 = group["betas"]
                opts = _OPTS.pack(_DT[dtype], _DT[kind], self.state_bits, group["lr"], beta1, beta2, group["eps"],
                                  group["weight_decay"], self.steps, scale)
                check(f(table.buffer_info()[0], len(table) // _FIELDS, opts, stream), "adamw_step")
        return loss

    def state_dict(self):
        d = super().state_dict()
        d["steps"] = self.steps
        return d

    def load_state_dict(self, state_dict):
        """Copies a state into the packed buffers (same parameters, same
        state_bits and master_weights)."""
        every = [p for g in self.param_groups for p in g["params"]]
        ids = [i for g in state_dict["param_groups"] for i in g["params"]]
        if len(ids) != len(every) or [len(g["params"]) for g in state_dict["param_groups"]] != \
                [len(g["params"]) for g in self.param_groups]:
            raise ValueError("the state is of other parameters")
        for i, p in zip(ids, every):
            theirs, mine = state_dict["state"].get(i, {}), self.state[p]
            if set(theirs) != set(mine) or any(theirs[k].shape != v.shape or theirs[k].dtype != v.dtype
                                               for k, v in mine.items()):
                raise ValueError("the state does not fit: other shapes, state_bits or master_weights")
        for i, p in zip(ids, every):
            for k, v in self.state[p].items():
                v.copy_(state_dict["state"][i][k])
        for g, new in zip(self.param_groups, state_dict["param_groups"]):
            g.update({k: v for k, v in new.items() if k != "params"})
        self.steps = state_dict["steps"]
