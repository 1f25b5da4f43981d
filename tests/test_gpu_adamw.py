"""GPU parity of the AdamW step: the moments and their 8-bit codes and scales
bit for bit against the same fp32 operations in numpy, the weights against
float64.

The weights' tolerance: the update is a product of five fp32 factors with a
root and a quotient, each within 2 units of 2^-24 (16 in all), the decay and
the difference are 2 roundings of the weight, and a stored weight is off by
half a step of its type.
"""
import ctypes

import numpy as np
import pytest
import torch

from birkhoff_projection_gb300 import _DT, _lib, optim
from oracle import block as ob

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, H = torch.float32, torch.bfloat16
HYPER = dict(lr=0.01, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.1)
SHAPES = [(300, 7), (1,), (128,), (127,), (129,), (2048,), (4097,), (64, 64), (0,), (5, 3, 3)]


def rnd(seed, *shape, std=1.0):
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(*shape, generator=g) * std
    return x * torch.exp(2 * torch.randn(*shape, generator=g))


def f32(t):
    return t.detach().float().cpu().numpy().ravel()


class Twin:
    """The same parameters in numpy."""

    def __init__(self, params, bits, master):
        self.bits, self.master = bits, master
        self.p = [f32(p) for p in params]
        z = [np.zeros(q.size, np.float32) for q in self.p]
        self.m = [ob.encode(q, False) for q in z] if bits == 8 else z
        self.v = [ob.encode(q, True) for q in z] if bits == 8 else [q.copy() for q in z]
        self.step_no = 0

    def step(self, params, opt, grads, lr, betas, eps, weight_decay, grad_scale=None):
        """Takes the step in numpy and compares everything."""
        self.step_no += 1
        for k, (p, g) in enumerate(zip(params, grads)):
            if g is None:
                continue
            m, v = self.m[k], self.v[k]
            if self.bits == 8:
                root = ob.decode(*v)
                m, v = ob.decode(*m), root * root
            m, v = ob.adamw_moments(f32(g), m, v, *betas, grad_scale)
            old = self.p[k]
            new, size = ob.adamw_weights(old, m, v, self.step_no, lr, *betas, eps, weight_decay)
            state = opt.state[p]
            held = f32(state["master"]) if self.master else f32(p)
            half = 0.0 if self.master else torch.finfo(p.dtype).eps / 2
            lim = 2.0 ** -24 * (16 * size + 3 * np.abs(old)) + half * np.abs(new) + 1e-37
            assert (np.abs(held - new) <= lim).all(), (k, np.max(np.abs(held - new) / lim))
            if self.master:  # the parameter is its master's nearest bf16
                assert torch.equal(p.detach(), state["master"].to(p.dtype))
            self.p[k] = held
            if self.bits == 8:
                self.m[k], self.v[k] = ob.encode(m, False), ob.encode(np.sqrt(v), True)
                for name, want in (("exp_avg", self.m[k]), ("exp_avg_sq_root", self.v[k])):
                    assert np.array_equal(f32(state[name]), want[0].astype(np.float32)), (k, name)
                    assert np.array_equal(f32(state[name + "_scale"]), want[1]), (k, name)
            else:
                self.m[k], self.v[k] = m, v
                assert np.array_equal(f32(state["exp_avg"]), m) and np.array_equal(f32(state["exp_avg_sq"]), v), k


def make(shapes, dtype, bits, master, seed=0, **how):
    params = [torch.nn.Parameter(rnd(seed + k, *s).to(dtype).to(DEV)) for k, s in enumerate(shapes)]
    return params, optim.AdamW(params, state_bits=bits, master_weights=master, **{**HYPER, **how})


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dtype,gtype,master", [(F, F, False), (F, H, False), (H, H, False), (H, F, False), (H, H, True),
                                                (H, F, True)])
def test_steps(dtype, gtype, master, bits):
    params, opt = make(SHAPES, dtype, bits, master)
    twin = Twin(params, bits, master)
    for t in range(4):
        grads = [rnd(100 * t + k, *s, std=0.1).to(gtype).to(DEV) for k, s in enumerate(SHAPES)]
        if dtype == gtype:
            for p, g in zip(params, grads):
                p.grad = g
            opt.step()
        else:  # a parameter's .grad has its type: the C entry takes any pair
            (_, _, some, rows, _), = opt._plans
            some_grads = [g for g in grads if g.numel()]
            table = (_lib.AdamwTensor * len(some))(*[
                _lib.AdamwTensor(p.data_ptr(), g.data_ptr(), *rows[8 * k + 2:8 * k + 8])
                for k, (p, g) in enumerate(zip(some, some_grads))])
            o = _lib.AdamwOpts(_DT[dtype], _DT[gtype], bits, HYPER["lr"], *HYPER["betas"], HYPER["eps"],
                               HYPER["weight_decay"], t + 1, None)
            _lib.check(_lib.lib().adamw_step(table, len(table), ctypes.byref(o), None), "adamw_step")
            torch.cuda.synchronize()
        twin.step(params, opt, grads, **HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_missing_gradients_scale_and_zero_gradients(bits):
    params, opt = make(SHAPES, F, bits, False)
    twin = Twin(params, bits, False)
    scale = torch.tensor(0.37, device=DEV)
    for t in range(3):
        grads = [None if (k + t) % 3 == 0 else rnd(9 * t + k, *s).to(DEV) * (k % 2) for k, s in enumerate(SHAPES)]
        for p, g in zip(params, grads):
            p.grad = g
        opt.step(grad_scale=scale)
        twin.step(params, opt, grads, grad_scale=np.float32(0.37), **HYPER)


@pytest.mark.parametrize("bits", [32, 8])
def test_tensors_off_16_byte_boundaries(bits):
    """Parameters and gradients that are views at odd offsets of one buffer."""
    flat, gflat = rnd(1, 5000).to(DEV), rnd(2, 5000).to(DEV)
    places = [(1, 700), (703, 129), (1001, 1000), (2048, 1024), (4095, 905)]
    params = [torch.nn.Parameter(flat[a:a + n]) for a, n in places]
    opt = optim.AdamW(params, state_bits=bits, **HYPER)
    twin = Twin(params, bits, False)
    outside = torch.ones(5000, dtype=torch.bool, device=DEV)
    for a, n in places:
        outside[a:a + n] = False
    before = flat.clone()
    grads = [gflat[a:a + n] for a, n in places]
    for p, g in zip(params, grads):
        p.grad = g
    opt.step()
    twin.step(params, opt, grads, **HYPER)
    assert torch.equal(flat[outside], before[outside])


def test_more_tensors_than_one_launch_holds_and_groups():
    shapes = [(3 + k % 50,) for k in range(600)]
    params = [torch.nn.Parameter(rnd(k, *s).to(DEV)) for k, s in enumerate(shapes)]
    groups = [{"params": params[:250]}, {"params": params[250:], "weight_decay": 0.0, "lr": 0.5, "betas": (0.5, 0.8)}]
    opt = optim.AdamW(groups, **HYPER)
    a, b = Twin(params[:250], 32, False), Twin(params[250:], 32, False)
    for t in range(2):
        grads = [rnd(k + t, *s).to(DEV) for k, s in enumerate(shapes)]
        for p, g in zip(params, grads):
            p.grad = g
        opt.step()
        a.step(params[:250], opt, grads[:250], **HYPER)
        b.step(params[250:], opt, grads[250:], lr=0.5, betas=(0.5, 0.8), eps=1e-8, weight_decay=0.0)


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("hyper", [dict(lr=0.0), dict(betas=(0.0, 0.0)), dict(eps=0.1), dict(weight_decay=0.0, lr=1.0)])
def test_hyperparameters(bits, hyper):
    how = {**HYPER, **hyper}
    params, opt = make([(1000,)], F, bits, False, **how)
    twin = Twin(params, bits, False)
    for t in range(2):
        params[0].grad = rnd(5 + t, 1000).to(DEV)
        opt.step()
        twin.step(params, opt, [params[0].grad], **how)


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_a_gradient_that_is_not_finite_stays_at_its_element(bad):
    for bits in (32, 8):
        a, oa = make([(1000,)], F, bits, False)
        b, ob_ = make([(1000,)], F, bits, False)
        g = rnd(3, 1000).to(DEV)
        b[0].grad = g.clone()
        g[200] = bad
        a[0].grad = g
        g[130] = b[0].grad[130] = 1e3  # the block's largest, so that its scale is the same without the bad one
        oa.step(), ob_.step()
        rest = torch.arange(1000, device=DEV) != 200
        assert torch.equal(a[0].detach()[rest], b[0].detach()[rest])
        for k, v in oa.state[a[0]].items():
            w = ob_.state[b[0]][k].float()
            assert torch.equal(v.float()[rest] if v.numel() == 1000 else v.float(), w[rest] if v.numel() == 1000 else w), k
        m = oa.state[a[0]]["exp_avg"].float()[200]
        assert not torch.isfinite(m) and not torch.isfinite(a[0][200])


def test_tiny_and_huge_gradients():
    """Magnitudes at the ends of fp32: squares that underflow or overflow, and
    blocks whose largest is subnormal."""
    for bits in (32, 8):
        for size in (1e-44, 1e-38, 1e-30, 1e-22, 1e15, 1e19):
            params, opt = make([(300,)], F, bits, False)
            twin = Twin(params, bits, False)
            g = (torch.linspace(-1, 1, 300) * size).to(DEV)
            params[0].grad = g
            opt.step()
            twin.step(params, opt, [g], **HYPER)


def test_a_weight_near_its_optimum_converges_in_8_bits():
    """Least squares in 8 bits follows 32 bits."""
    target = rnd(1, 4096).clamp(-3, 3).to(DEV)
    loss = {}
    for bits in (32, 8):
        p = torch.nn.Parameter(torch.zeros(4096, device=DEV))
        opt = optim.AdamW([p], lr=0.02, betas=(0.9, 0.95), weight_decay=0.0, state_bits=bits)
        for _ in range(400):
            p.grad = p.detach() - target
            opt.step()
        loss[bits] = (p.detach() - target).square().mean().item()
    start = target.square().mean().item()
    assert loss[32] < 1e-3 * start and loss[8] < 1e-3 * start


@pytest.mark.parametrize("bits", [32, 8])
def test_state_round_trip(bits):
    a, oa = make([(300,), (64, 9)], H, bits, True)
    b, ob_ = make([(300,), (64, 9)], H, bits, True, seed=50)
    for t in range(3):
        for k, p in enumerate(a):
            p.grad = rnd(k + t, *p.shape).to(H).to(DEV)
        oa.step()
    with torch.no_grad():
        for p, q in zip(a, b):
            q.copy_(p)
    where = {k: v.data_ptr() for k, v in ob_.packed().items()}
    ob_.load_state_dict(oa.state_dict())
    assert ob_.steps == 3 and {k: v.data_ptr() for k, v in ob_.packed().items()} == where
    for k, (p, q) in enumerate(zip(a, b)):
        p.grad = rnd(80 + k, *p.shape).to(H).to(DEV)
        q.grad = p.grad.clone()
    oa.step(), ob_.step()
    assert all(torch.equal(p, q) for p, q in zip(a, b))
    other = make([(300,), (64, 9)], H, 40 - bits, True)[1]
    with pytest.raises(ValueError, match="fit"):
        other.load_state_dict(oa.state_dict())
    with pytest.raises(ValueError, match="other parameters"):
        make([(300,)], H, bits, True)[1].load_state_dict(oa.state_dict())


def test_refusals():
    with pytest.raises(TypeError):
        optim.AdamW([torch.nn.Parameter(torch.zeros(3, dtype=torch.half, device=DEV))])
    with pytest.raises(ValueError, match="contiguous"):
        optim.AdamW([torch.nn.Parameter(torch.zeros(4, 4, device=DEV).t()[:, :2])])
    with pytest.raises(ValueError, match="master"):
        optim.AdamW([torch.nn.Parameter(torch.zeros(3, device=DEV))], master_weights=True)
    params, opt = make([(4,)], F, 32, False)
    with pytest.raises(ValueError, match="construction"):
        opt.add_param_group({"params": [torch.nn.Parameter(torch.zeros(3, device=DEV))]})
    params[0].grad = torch.ones(4, device=DEV)
    with pytest.raises(ValueError, match="grad_scale"):
        opt.step(grad_scale=torch.ones(2, device=DEV))
    before = params[0].detach().clone()
    opt.param_groups[0]["lr"] = -1.0
    with pytest.raises(Exception, match="invalid"):
        opt.step()
    assert torch.equal(params[0].detach(), before) and opt.steps == 0
    opt.param_groups[0]["lr"] = 1.0
    params[0].data = torch.zeros(5, device=DEV)
    params[0].grad = torch.ones(5, device=DEV)
    with pytest.raises(ValueError, match="construction"):
        opt.step()


def test_a_bad_group_stops_every_group():
    params = [torch.nn.Parameter(torch.ones(9, device=DEV)) for _ in range(2)]
    opt = optim.AdamW([{"params": params[:1]}, {"params": params[1:]}])
    for p in params:
        p.grad = torch.ones(9, device=DEV)
    opt.param_groups[1]["betas"] = (0.9, 1.5)
    with pytest.raises(ValueError, match="betas"):
        opt.step()
    assert all((p == 1).all() for p in params) and opt.steps == 0


def test_gradients_that_are_not_contiguous():
    p = torch.nn.Parameter(rnd(1, 6, 8).to(DEV))
    q = torch.nn.Parameter(p.detach().clone())
    a, b = optim.AdamW([p], **HYPER), optim.AdamW([q], **HYPER)
    g = rnd(2, 8, 6).to(DEV)
    p.grad, q.grad = g.t(), g.t().contiguous()
    assert not p.grad.is_contiguous()
    a.step(), b.step()
    assert torch.equal(p, q)


def test_hooks_profiler_and_schedulers():
    p = torch.nn.Parameter(torch.ones(9, device=DEV))
    opt = optim.AdamW([p], lr=1.0)
    p.grad = torch.ones(9, device=DEV)
    seen = []
    handles = [opt.register_step_pre_hook(lambda *a: seen.append("before")), opt.register_step_post_hook(lambda *a: seen.append("after"))]
    opt.step()
    assert seen == ["before", "after"] and opt.steps == 1
    for h in handles:
        h.remove()
    sched = torch.optim.lr_scheduler.LambdaLR(opt, lambda n: 0.5 ** n)
    before = p.detach().clone()
    assert opt.step(lambda: torch.tensor(3.0)) == 3.0
    sched.step()
    assert opt.param_groups[0]["lr"] == 0.5 and opt.steps == 2 and not torch.equal(p, before) and len(seen) == 2
    with torch.profiler.profile(activities=[torch.profiler.ProfilerActivity.CPU]) as prof:
        opt.step()
    assert any("AdamW.step" in e.key for e in prof.key_averages()) and opt.steps == 3


def test_captured_in_a_graph():
    params, opt = make([(5000,), (64, 64)], F, 8, False)
    twins, other = make([(5000,), (64, 64)], F, 8, False)
    for k, (p, q) in enumerate(zip(params, twins)):
        p.grad = rnd(k, *p.shape).to(DEV)
        q.grad = p.grad.clone()
    g = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(g):
        opt.step()
    g.replay()
    other.step()
    torch.cuda.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(params, twins))
