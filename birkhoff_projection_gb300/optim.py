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
from collections import defaultdict

import torch
from torch.optim import optimizer as _hooks

from . import _DT
from ._lib import ADAMW_BLOCK, binding, check, lib

__all__ = ["AdamW"]

# adamw_tensor is eight 8-byte fields: p g m v m_scale v_scale master n
_FIELDS = 8
# adamw_opts: p_dtype g_dtype state_bits; lr beta1 beta2 eps weight_decay; step, grad_scale
_OPTS = struct.Struct("<3i4x5dqQ")


def _bytes(t):
    return t.view(torch.uint8) if t.dtype == torch.float8_e4m3fn else t


class AdamW(torch.optim.Optimizer):
    """AdamW with decoupled weight decay, one launch for up to 256 tensors of
    a group.

    params: fp32 or bf16 CUDA parameters, contiguous, on one device; a group
    may set its own lr, betas, eps and weight_decay.  state_bits: 32 or 8.
    master_weights: keep an fp32 copy of bf16 parameters and step on that.
    step(grad_scale=t) multiplies every gradient by the fp32 device scalar t.
    Autograd knows of a step as of any change in place: a graph that keeps the
    old parameters is refused by backward.
    A parameter without a gradient is left alone, and so are its moments; all
    parameters share one count of steps (the attribute `steps`).  The count and
    the group's numbers are arguments of the launch: a step captured into a CUDA
    graph repeats that very step.  copy.deepcopy and pickle of the optimizer
    together with its parameters give one that goes on by itself."""

    def __init__(self, params, lr: float = 1e-3, betas=(0.9, 0.999), eps: float = 1e-8, weight_decay: float = 1e-2, *,
                 state_bits: int = 32, master_weights: bool = False):
        self._check(lr, betas, eps, weight_decay)
        if state_bits not in (8, 32):
            raise ValueError("state_bits must be 8 or 32, got %r" % (state_bits,))
        self.steps = 0
        self.state_bits, self.master_weights = state_bits, bool(master_weights)
        self._packed, self._ready = None, False
        super().__init__(params, dict(lr=lr, betas=tuple(betas), eps=eps, weight_decay=weight_decay))
        self._ready = True
        self._pack()

    @staticmethod
    def _check(lr, betas, eps, weight_decay):
        inf = float("inf")
        if not (0.0 <= lr < inf and 0.0 <= eps < inf and 0.0 <= weight_decay < inf):
            raise ValueError("invalid lr, eps or weight_decay (finite and not negative): %r, %r, %r"
                             % (lr, eps, weight_decay))
        if len(betas) != 2 or not (0.0 <= betas[0] < 1.0 and 0.0 <= betas[1] < 1.0):
            raise ValueError("betas must be two numbers in [0, 1), got %r" % (betas,))

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
                self._plans.append((group, dtype, params, rows, rows.tobytes()))

    def packed(self) -> dict:
        """The packed state buffers: exp_avg and exp_avg_sq (32 bits), or
        exp_avg and exp_avg_sq_root as e4m3 with exp_avg_scale and
        exp_avg_sq_root_scale (8 bits); master with master weights.  The
        tensors follow each other in the order of the parameters, each on a
        multiple of 128 elements."""
        return dict(self._packed)

    def step(self, closure=None, *, grad_scale: torch.Tensor = None):
        """One step on the parameters' gradients (fp32 or bf16, contiguous)."""
        # torch's wrapper of a step, for its hooks and the profiler's mark, takes
        # longer than a small step: only where there is use for it
        if (self._optimizer_step_pre_hooks or self._optimizer_step_post_hooks or _hooks._global_optimizer_pre_hooks
                or _hooks._global_optimizer_post_hooks or torch.autograd._profiler_enabled()):
            return self._marked_step(self, closure, grad_scale=grad_scale)
        return self._step(closure, grad_scale=grad_scale)

    step.hooked = True  # torch.optim.Optimizer leaves it as it is

    def _step(self, closure=None, *, grad_scale=None):
        loss = None
        if closure is not None:
            with torch.enable_grad():
                loss = closure()
        if grad_scale is not None and (grad_scale.dtype != torch.float32 or grad_scale.numel() != 1
                                       or grad_scale.device != self._device):
            raise ValueError("grad_scale must be one float32 on %s" % self._device)
        dev = self._device.index
        calls = []  # the tables, the parameters in them, and whatever they point to that is not kept elsewhere
        plain = binding().adamw_table
        for group, dtype, params, rows, packed in self._plans:
            got = plain(params, packed, _DT[dtype], dev)  # None where the gradients are not all plain
            if got is not None:
                calls.append((group, _DT[dtype], got[1], got[0], params, None))
                continue
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
            for k, (p, g) in enumerate(zip(params, grads)):
                if p.dtype != dtype or p.get_device() != dev or not p.is_contiguous() \
                        or not p.numel() == g.numel() == rows[(k + 1) * _FIELDS - 1]:
                    raise ValueError("parameters must stay as they were at construction: contiguous, of one type and "
                                     "size, on %s" % self._device)
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
                    theirs = [p for p, g in zip(params, grads) if g.dtype == kind]
                else:
                    mine, theirs = table, params
                calls.append((group, _DT[dtype], _DT[kind], mine.tobytes(), theirs, grads))
        for group, *_ in calls:  # before the first launch
            self._check(group["lr"], group["betas"], group["eps"], group["weight_decay"])
        scale = 0 if grad_scale is None else grad_scale.data_ptr()
        if dev == torch.cuda.current_device():
            self._launch(calls, scale)
        else:
            with torch.cuda.device(dev):
                self._launch(calls, scale)
        self.steps += 1
        return loss

    def _launch(self, calls, scale):
        f, stream = lib().adamw_step, torch._C._cuda_getCurrentRawStream(self._device.index)
        for group, p_type, g_type, table, params, _ in calls:
            beta1, beta2 = group["betas"]
            opts = _OPTS.pack(p_type, g_type, self.state_bits, group["lr"], beta1, beta2, group["eps"],
                              group["weight_decay"], self.steps + 1, scale)
            check(f(table, len(table) // (8 * _FIELDS), opts, stream), "adamw_step")
            # the kernel writes by address: autograd is told, so that a graph which
            # keeps the old values is refused
            torch.autograd.graph.increment_version(params)

    _marked_step = staticmethod(torch.optim.Optimizer.profile_hook_step(_step))

    def __getstate__(self):
        """For copy.deepcopy and pickle, with the parameters.  The state goes
        as its packed buffers (a parameter's views would each take all of one
        along), e4m3 numbers as bytes (not every pickle has the type)."""
        return {**super().__getstate__(), "state": {}, "steps": self.steps, "state_bits": self.state_bits,
                "master_weights": self.master_weights, "_packed": {k: _bytes(t) for k, t in self._packed.items()}}

    def __setstate__(self, state):
        super().__setstate__(state)
        packed, self.state = self._packed, defaultdict(dict)
        self._pack()
        for k, t in self._packed.items():
            _bytes(t).copy_(packed[k])
        self._ready = True

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
