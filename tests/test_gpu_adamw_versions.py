"""AdamW writes parameters in place, and autograd knows of it: a backward pass
through a graph from before the step is refused, as with torch's optimizers."""
import pytest
import torch

from birkhoff_projection_gb300 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def graph(p):
    return (p * p).sum()  # keeps p


@pytest.mark.parametrize("dtype,how", [(torch.float32, {}), (torch.bfloat16, {}), (torch.bfloat16, dict(master_weights=True)),
                                       (torch.float32, dict(state_bits=8))])
@pytest.mark.parametrize("plain", [True, False])
def test_an_old_graph_is_refused_after_the_step(dtype, how, plain):
    """plain: gradients as the short way from Python takes them; otherwise one
    is missing and one is not contiguous."""
    ps = [torch.nn.Parameter(torch.randn(6, 8, device=DEV).to(dtype)) for _ in range(3)]
    opt = optim.AdamW(ps, **how)
    losses = [graph(p) for p in ps]
    torch.autograd.backward(losses, retain_graph=True)
    if not plain:
        ps[1].grad = None
        ps[2].grad = ps[2].grad.t().contiguous().t()
        assert not ps[2].grad.is_contiguous()
    before = [p._version for p in ps]
    opt.step()
    for k, p in enumerate(ps):
        stepped = plain or k != 1
        assert (p._version > before[k]) == stepped
        if stepped:
            with pytest.raises(RuntimeError, match="modified by an inplace operation"):
                losses[k].backward()
        else:
            losses[k].backward()
    # a graph from behind the step is as good as ever
    graph(ps[0]).backward()


def test_a_refused_step_changes_no_version():
    p = torch.nn.Parameter(torch.ones(9, device=DEV))
    opt = optim.AdamW([p])
    p.grad = torch.ones(9, device=DEV)
    opt.param_groups[0]["lr"] = -1.0
    before = p._version
    with pytest.raises(ValueError):
        opt.step()
    assert p._version == before
