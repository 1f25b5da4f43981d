"""The example network: with the kernels and with plain operations in their
place, trained, and served token by token."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))
EPS = torch.finfo(torch.bfloat16).eps / 2


@pytest.fixture(scope="module")
def example():
    path = os.path.join(os.path.dirname(HERE), "examples", "hyper_connections.py")
    spec = importlib.util.spec_from_file_location("hyper_connections", path)
    module = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(module)
    return module


def _norm(u, weight, eps=1e-6):
    u = u * torch.rsqrt((u * u).mean(-1, keepdim=True) + eps)
    return u if weight is None else u * weight.float()


def _enter(x, a, weight):
    u = x.float() if a is None else a.float()[..., None] * x.float()
    return _norm(u.sum(-2), weight).to(x.dtype)


def _leave(x, y, P, b, *, gate, act, weight):
    assert act == "sigmoid"
    v = torch.sigmoid(gate.float()) * _norm(y.float(), weight)
    return ((P.float() @ x.float()) + b.float()[..., None] * v[..., None, :]).to(x.dtype)


def _leave_enter(x, y, P, b, *, gate, act, weight, a_next, weight_next):
    out = _leave(x, y, P, b, gate=gate, act=act, weight=weight)
    return out, _enter(out, a_next, weight_next)


def _network(example, blocks, width):
    torch.manual_seed(1)
    return example.Network(width=width, blocks=blocks).to("cuda", torch.bfloat16)


@pytest.mark.parametrize("blocks,width", [(1, 64), (2, 128), (2, 100)])
def test_with_plain_operations(example, monkeypatch, blocks, width):
    """Logits and gradients.  Both sides round at the same places, and differ
    where another order of sums in fp32 lets a rounding to bf16 fall the other
    way: at most a step of 2 EPS each.  Rounded on the way through a block are
    its input, two halves and the product of the MLP, y, the gate, the
    coefficients and the streams, 8 values, and at the ends the embedding, h
    and the logits, 3; a gradient takes the way twice."""
    net = _network(example, blocks, width)
    tokens = example.Chain(16, "cuda").sample(3, 17)
    got = []
    for plain in (False, True):
        if plain:
            for name, f in (("enter", _enter), ("leave", _leave), ("leave_enter", _leave_enter)):
                monkeypatch.setattr(example, name, f)
        net.zero_grad()
        logits = net(tokens[:, :-1])
        torch.nn.functional.cross_entropy(logits.flatten(0, 1), tokens[:, 1:].flatten()).backward()
        got.append([logits.detach()] + [p.grad.float() for p in net.parameters()])
    rounded = 8 * blocks + 3
    for k, (mine, theirs) in enumerate(zip(*got)):
        bound = (rounded if k == 0 else 2 * rounded) * 2 * EPS
        assert torch.isfinite(mine).all()
        assert (mine - theirs).norm() <= bound * theirs.norm(), k


def test_served_as_trained(example):
    """A token at a call gives what the whole sequence gives, up to the
    roundings counted above."""
    net = _network(example, 2, 96)
    tokens = example.Chain(16, "cuda").sample(5, 11)
    with torch.no_grad():
        whole = net(tokens)
        out, logits = example.serve(net, tokens, 0)
    assert torch.equal(out, tokens)
    assert (logits - whole).norm() <= 19 * 2 * EPS * whole.norm()


def test_training_and_serving(example, capsys):
    """The loss begins near ln 16 = 2.77 and has the chain's entropy, at most
    ln 4 = 1.39, below it.  Of one known symbol the next keeps more than 2:
    64 draws of 16 are behind it."""
    losses, right = example.main(["--steps", "120", "--width", "256", "--blocks", "2"])
    assert losses[0] > 2.5 and losses[-1] < 2.0
    assert right > 0.5
    assert "served" in capsys.readouterr().out
