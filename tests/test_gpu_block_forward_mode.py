"""Forward-mode differentiation: the block operators have no such derivative,
and say so instead of returning a result without a tangent (which the rest of
a graph would read as a derivative of zero)."""
import pytest
import torch
import torch.autograd.forward_ad as fwad

import birkhoff_projection_gb300 as b4
from birkhoff_projection_gb300 import block

pytestmark = pytest.mark.gpu
T, S, C = 3, 4, 24


def tensors(spread):
    """All tensors of the calls; spread: views that are not contiguous."""
    g = torch.Generator().manual_seed(0)

    def some(*shape):
        t = torch.randn(*shape, 2 if spread else 1, generator=g).to("cuda:0")
        return t[..., 0] if spread else t.squeeze(-1)

    return dict(x=some(T, S, C), y=some(T, C), P=some(T, S, S), b=some(T, S), gate=some(T, C), w=some(C), a=some(T, S),
                w2=some(C), dout=some(T, S, C), dh=some(T, C), out=some(T, S, C))


CALLS = {
    "enter": ("x a w", lambda k: block.enter(k["x"], k["a"], k["w"])),
    "leave": ("x y P b gate w", lambda k: block.leave(k["x"], k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"])),
    "leave_enter": ("x y P b gate w a w2", lambda k: block.leave_enter(
        k["x"], k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"], a_next=k["a"], weight_next=k["w2"])),
    "enter_backward": ("dh x a w dout", lambda k: block.enter_backward(k["dh"], k["x"], k["a"], k["w"], dres=k["dout"])),
    "leave_backward": ("dout x y P b gate w", lambda k: block.leave_backward(
        k["dout"], k["x"], k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"])),
    "leave_enter_backward": ("dout dh out x y P b gate w a w2", lambda k: block.leave_enter_backward(
        k["dout"], k["dh"], k["out"], k["x"], k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"], a_next=k["a"],
        weight_next=k["w2"])),
}


@pytest.mark.parametrize("grad", [True, False])
@pytest.mark.parametrize("spread", [False, True])
@pytest.mark.parametrize("name", sorted(CALLS))
def test_a_tangent_is_refused(name, spread, grad):
    which, call = CALLS[name]
    plain = tensors(spread)
    for n in which.split():
        with fwad.dual_level(), torch.set_grad_enabled(grad):
            k = dict(plain)
            k[n] = fwad.make_dual(k[n], torch.ones_like(k[n]))
            with pytest.raises(NotImplementedError):
                call(k)
            call(plain)  # a level alone is no tangent
    call(plain)


def test_a_tangent_of_the_gradient_is_refused():
    """Forward over reverse."""
    k = tensors(False)
    x = k["x"].clone().requires_grad_()
    h = block.enter(x, k["a"], k["w"])
    with fwad.dual_level():
        with pytest.raises(NotImplementedError):
            torch.autograd.grad(h, x, fwad.make_dual(k["dh"], torch.ones_like(k["dh"])))


def test_the_projection_refuses_it_too():
    X = torch.randn(5, 4, 4, device="cuda:0")
    with fwad.dual_level(), pytest.raises(NotImplementedError):
        b4.project(fwad.make_dual(X, torch.ones_like(X)))
