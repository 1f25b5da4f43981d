"""Autograd computes the gradients that somebody asks for: each alone is the
one that all of them together give, and no room is taken for the others."""
import pytest
import torch

from birkhoff_projection_gb300 import block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, H = torch.float32, torch.bfloat16


def make(T, S, C, dtype, spread=False):
    g = torch.Generator().manual_seed(3)

    def some(*shape, t=dtype):
        v = torch.randn(*shape, 2 if spread else 1, generator=g).to(t).to(DEV)
        return v[..., 0] if spread else v.squeeze(-1)

    k = dict(x=some(T, S, C), y=some(T, C), b=some(T, S, t=F), gate=some(T, C), weight=some(C, t=F), a_next=some(T, S, t=F),
             weight_next=some(C, t=F))
    k["P"] = some(T, S, S, t=F) if S > 1 else None
    return k, some(T, S, C), some(T, C)


def call(name, k):
    if name == "enter":
        return [block.enter(k["x"], k["a_next"], k["weight_next"])]
    how = dict(gate=k["gate"], act="silu", weight=k["weight"], scale=0.3)
    if name == "leave":
        return [block.leave(k["x"], k["y"], k["P"], k["b"], **how)]
    return block.leave_enter(k["x"], k["y"], k["P"], k["b"], a_next=k["a_next"], weight_next=k["weight_next"], **how)


def gradients(name, k, which, dout, dh, use="both"):
    """The gradients of the tensors `which`; use: the results that the loss has."""
    k = {n: t if t is None else t.detach().requires_grad_(n in which) for n, t in k.items()}
    got = call(name, k)
    up = [dh] if name == "enter" else [dout] if name == "leave" else [dout, dh]
    if use != "both":
        n = ("out", "h").index(use)
        got, up = got[n:n + 1], up[n:n + 1]
    torch.autograd.backward(got, up)
    return {n: k[n].grad for n in which}


TENSORS = {"enter": ["x", "a_next", "weight_next"], "leave": ["x", "y", "P", "b", "gate", "weight"],
           "leave_enter": ["x", "y", "P", "b", "gate", "weight", "a_next", "weight_next"]}


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("S,C", [(4, 264), (1, 512), (3, 77)])
@pytest.mark.parametrize("name", sorted(TENSORS))
def test_each_alone(name, S, C, spread, dtype):
    k, dout, dh = make(9, S, C, dtype, spread)
    every = [n for n in TENSORS[name] if k[n] is not None]
    want = gradients(name, k, every, dout, dh)
    for n in every:
        got = gradients(name, k, [n], dout, dh)
        assert torch.equal(got[n], want[n]), n
    pair = every[::2]
    got = gradients(name, k, pair, dout, dh)
    assert all(torch.equal(got[n], want[n]) for n in pair)


@pytest.mark.parametrize("dtype", [F, H])
@pytest.mark.parametrize("S,C", [(4, 264), (1, 512), (3, 77)])
def test_one_result_of_two(S, C, dtype):
    """leave_enter of which the loss has one result: leave's gradients, or those with a zero for the other."""
    k, dout, dh = make(9, S, C, dtype)
    every = [n for n in TENSORS["leave_enter"] if k[n] is not None]
    got = gradients("leave_enter", k, every, dout, dh, "out")
    want = gradients("leave", k, [n for n in every if not n.endswith("next")], dout, dh)
    assert all(torch.equal(got[n], want[n]) for n in want)
    assert all(got[n] is None or not got[n].any() for n in every if n.endswith("next"))
    got = gradients("leave_enter", k, every, dout, dh, "h")
    want = gradients("leave_enter", k, every, torch.zeros_like(dout), dh)
    assert all(torch.equal(got[n], want[n]) for n in every)


def room(name, k, which, dout, dh, use="both"):
    """Bytes that a backward pass takes at most beside what there is before it."""
    k = {n: t if t is None else t.detach().requires_grad_(n in which) for n, t in k.items()}
    got = call(name, k)
    up = [dh] if name == "enter" else [dout] if name == "leave" else [dout, dh]
    if use != "both":
        n = ("out", "h").index(use)
        got, up = got[n:n + 1], up[n:n + 1]
    torch.cuda.synchronize()
    torch.cuda.reset_peak_memory_stats()
    before = torch.cuda.memory_allocated()
    torch.autograd.backward(got, up)
    return torch.cuda.max_memory_allocated() - before


def test_no_room_for_the_others():
    T, S, C = 2048, 4, 1024
    k, dout, dh = make(T, S, C, F)
    streams, row = dout.numel() * 4, dh.numel() * 4  # 32 MB and 8 MB
    few = row // 2  # a weight's partial sums, coefficients
    assert room("enter", k, ["a_next"], dout, dh) < few
    assert room("leave", k, ["P"], dout, dh) < few
    assert room("leave", k, ["y"], dout, dh) < row + few
    assert room("leave", k, ["x"], dout, dh) < streams + few
    # h alone: the gradient of the streams, and no zeros for that of `out`
    assert room("leave_enter", k, ["a_next", "P"], dout, dh, "h") < streams + few
