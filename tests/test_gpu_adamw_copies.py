"""copy.deepcopy and pickle of the optimizer with its parameters: the copy
steps on its own parameters and state, from where the original was."""
import copy
import io
import pickle

import pytest
import torch

from birkhoff_projection_gb300 import optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def through_pickle(both):
    f = io.BytesIO()
    pickle.dump(both, f)
    f.seek(0)
    return pickle.load(f)


def through_torch(both):
    f = io.BytesIO()
    torch.save(both, f)
    f.seek(0)
    return torch.load(f, weights_only=False)


def gradients(params, seed):
    g = torch.Generator().manual_seed(seed)
    for p in params:
        p.grad = torch.randn(*p.shape, generator=g).to(p.dtype).to(DEV)


@pytest.mark.parametrize("bits,dtype,master", [(32, torch.float32, False), (8, torch.float32, False),
                                               (8, torch.bfloat16, True), (32, torch.bfloat16, True)])
@pytest.mark.parametrize("copied", [copy.deepcopy, through_pickle, through_torch])
def test_a_copy_goes_on_by_itself(copied, bits, dtype, master):
    torch.manual_seed(0)
    params = [torch.nn.Parameter(torch.randn(*s, device=DEV).to(dtype)) for s in ((300,), (64, 9), (0,), (1,))]
    opt = optim.AdamW([{"params": params[:1], "lr": 0.02}, {"params": params[1:]}], lr=0.01, weight_decay=0.1,
                      state_bits=bits, master_weights=master)
    for t in range(3):
        gradients(params, t)
        opt.step()
    twins, other = copied((params, opt))
    assert other.steps == 3 and other.state_bits == bits and other.master_weights == master
    assert [id(p) for g in other.param_groups for p in g["params"]] == [id(p) for p in twins]
    assert [g["lr"] for g in other.param_groups] == [0.02, 0.01]
    # all state is the copy's own, and consists of views of its packed buffers
    for name, buf in other.packed().items():
        assert torch.equal(buf.view(torch.uint8), opt.packed()[name].view(torch.uint8))
        assert buf.data_ptr() != opt.packed()[name].data_ptr()
        first, end = buf.data_ptr(), buf.data_ptr() + buf.numel() * buf.element_size()
        for q in twins:
            assert q.numel() == 0 or first <= other.state[q][name].data_ptr() < end
    # the copy's step leaves the original alone
    kept = [p.detach().clone() for p in params]
    state = {k: v.clone() for k, v in opt.packed().items()}
    gradients(twins, 7)
    other.step()
    assert other.steps == 4 and opt.steps == 3
    assert all(torch.equal(p, q) for p, q in zip(params, kept))
    assert all(torch.equal(v.view(torch.uint8), opt.packed()[k].view(torch.uint8)) for k, v in state.items())
    # and is the step that the original takes on the same gradients
    gradients(params, 7)
    opt.step()
    for p, q in zip(params, twins):
        assert torch.equal(p, q)
        for name in opt.state[p]:
            assert torch.equal(opt.state[p][name].float(), other.state[q][name].float()), name
    # a copy's state dictionary, and closures and hooks, work as they did
    again = optim.AdamW([{"params": twins[:1]}, {"params": twins[1:]}], state_bits=bits, master_weights=master)
    again.load_state_dict(other.state_dict())
    assert again.steps == 4 and other.step(lambda: 3.0) == 3.0
    with pytest.raises(ValueError, match="construction"):
        other.add_param_group({"params": [torch.nn.Parameter(torch.zeros(3, device=DEV))]})
