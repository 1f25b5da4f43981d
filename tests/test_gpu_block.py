"""GPU parity of the hyper-connection block operators (enter, leave,
leave_enter and their gradients) against the float64 oracle.

Tolerance, fixed from the kernels' arithmetic: a value is within
N 2^-24 of its magnitude (the oracle's sum of its terms' absolute values) plus
half a step of its own type.  N = 256: a sum over a row is at most 32
sequential additions in a thread, 5 in a warp and 16 over warps, each weight
gradient at most 40 + 16 more over CTAs, and a result multiplies up to three
such sums and a handful of rounded factors.  The 2-norm of the error is held
to 16 2^-24 of the magnitudes' (roundings of either sign: the root of N).
"""
import ctypes

import numpy as np
import pytest
import torch

import birkhoff_projection_gb300 as b4
from birkhoff_projection_gb300 import _lib, block
from oracle import block as ob

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, H = torch.float32, torch.bfloat16
TYPES = [(F, F), (H, H), (F, H)]
N = 256


def np64(t):
    return None if t is None else t.detach().double().cpu().numpy()


def rnd(seed, *shape, dtype=F, std=1.0, mean=0.0):
    g = torch.Generator().manual_seed(seed)
    return (torch.randn(*shape, generator=g) * std + mean).to(dtype).to(DEV)


def close(got, want, name=""):
    value, mag = want
    assert tuple(got.shape) == value.shape, name
    half = torch.finfo(got.dtype).eps / 2
    g = np64(got)
    assert np.isfinite(g).all(), name
    err, lim = np.abs(g - value), N * 2.0 ** -24 * mag + half * np.abs(value) + 1e-37
    assert (err <= lim).all(), "%s: %g of the limit at %s" % (name, (err / lim).max(), np.unravel_index((err / lim).argmax(), err.shape))
    norm = np.linalg.norm
    assert norm(err) <= 16 * 2.0 ** -24 * norm(mag) + half * norm(value) + 1e-37, name


def compare(got, want):
    for name, t in got._asdict().items():
        if t is not None:
            close(t, want[name], name)


def inputs(T, S, C, tx, ty, act="sigmoid", mix=True, coef=F, weight=F, seed=0):
    k = {"x": rnd(seed, T, S, C, dtype=tx), "y": rnd(seed + 1, T, C, dtype=ty, std=2.0)}
    k["P"] = torch.softmax(rnd(seed + 2, T, S, S), -1).to(coef) if mix else None
    k["b"] = rnd(seed + 3, T, S, dtype=coef) if mix else None
    k["gate"] = None if act is None else rnd(seed + 4, T, C, dtype=ty, std=2.0)
    k["w"] = rnd(seed + 5, C, dtype=weight, std=0.2, mean=1.0)
    k["a"] = rnd(seed + 6, T, S, dtype=coef) if mix else None
    k["w2"] = rnd(seed + 7, C, dtype=weight, std=0.2, mean=1.0)
    k["D"], k["dh"] = rnd(seed + 8, T, S, C, dtype=tx), rnd(seed + 9, T, C, dtype=ty)
    return k


def direct(entry, tensors, T, S, C, dtype, act=0):
    """A call of the C entry with contiguous tensors of one type, fp32 coefficients and weights."""
    kind = 1 if dtype == H else 0
    args = _lib.HcbArgs(T=T, S=S, C=C, x_dtype=kind, y_dtype=kind, act=act, norm=1, eps=1e-6, scale=1.0)
    for name, t in tensors.items():
        if t is not None:
            setattr(args, name, t.data_ptr())
    for name in ("x", "dout", "dres"):
        setattr(args, name + "_ts", S * C)
        setattr(args, name + "_ss", C)
    for name, n in (("y", C), ("gate", C), ("dh", C), ("P", S * S), ("a", S), ("b", S)):
        setattr(args, name + "_ts", n)
    if tensors.get("workspace") is not None:
        args.workspace_bytes = tensors["workspace"].numel()
    _lib.check(getattr(_lib.lib(), entry)(ctypes.byref(args), torch.cuda.current_stream().cuda_stream), entry)


def everything(k, act="sigmoid", norm=True, scale=0.5, eps=1e-6, eps2=1e-5):
    """All six functions on one set of inputs, each against the oracle."""
    n = {name: np64(t) for name, t in k.items()}
    ty = k["y"].dtype
    close(block.enter(k["x"], k["a"], k["w"], eps=eps, out_dtype=ty), ob.enter(n["x"], n["a"], n["w"], eps)["h"], "h")
    compare(block.enter_backward(k["dh"], k["x"], k["a"], k["w"], eps=eps, dres=k["D"]),
            ob.enter_backward(n["dh"], n["x"], n["a"], n["w"], eps, n["D"]))
    how = dict(act=act, norm=norm, scale=scale, eps=eps)
    mine = dict(gate=k["gate"], weight=k["w"], **how)
    theirs = dict(gate=n["gate"], w=n["w"], **how)
    want = ob.leave(n["x"], n["y"], n["P"], n["b"], **theirs)["out"]
    close(block.leave(k["x"], k["y"], k["P"], k["b"], **mine), want, "out")
    compare(block.leave_backward(k["D"], k["x"], k["y"], k["P"], k["b"], **mine),
            ob.leave_backward(n["D"], n["x"], n["y"], n["P"], n["b"], **theirs))
    out, h = block.leave_enter(k["x"], k["y"], k["P"], k["b"], a_next=k["a"], weight_next=k["w2"], eps_next=eps2, **mine)
    close(out, want, "out")
    # h is of the streams as they are stored
    close(h, ob.enter(np64(out), n["a"], n["w2"], eps2)["h"], "h after leave")
    compare(block.leave_enter_backward(k["D"], k["dh"], out, k["x"], k["y"], k["P"], k["b"], a_next=k["a"],
                                       weight_next=k["w2"], eps_next=eps2, **mine),
            ob.leave_enter_backward(n["D"], n["dh"], np64(out), n["x"], n["y"], n["P"], n["b"], a_next=n["a"],
                                    w_next=n["w2"], eps_next=eps2, **theirs))


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("S", [1, 2, 3, 4, 5, 8])
@pytest.mark.parametrize("T,C", [(1, 1), (3, 7), (130, 64), (5, 1000), (2, 1001), (300, 520)])
def test_all_operators(T, S, C, tx, ty):
    everything(inputs(T, S, C, tx, ty, seed=T + S + C))


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("T,S,C", [(1, 4, 4096), (700, 4, 2048), (3, 1, 16384), (3, 4, 16384), (2, 8, 16384), (2, 2, 16383),
                                   (1500, 1, 256), (2000, 4, 40), (160, 4, 5120)])
def test_long_rows_and_many_tokens(T, S, C, tx, ty):
    everything(inputs(T, S, C, tx, ty, seed=3))


@pytest.mark.parametrize("act", [None, "sigmoid", "silu", "linear"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("mix", [True, False])
def test_gates_norm_and_mixing(act, norm, mix):
    for S, C, (tx, ty) in ((4, 264, (H, H)), (1, 100, (F, F)), (3, 77, (F, H))):
        everything(inputs(9, S, C, tx, ty, act, mix), act or "sigmoid", norm, scale=-1.25, eps=1e-3)


def test_bf16_coefficients_and_weights():
    everything(inputs(9, 4, 264, H, H, coef=H, weight=H))
    everything(inputs(9, 3, 33, F, F, coef=H, weight=H))


def test_without_weights_and_coefficients():
    k = inputs(6, 4, 72, F, F, act=None, mix=False)
    k["w"] = k["w2"] = None
    everything(k)


@pytest.mark.parametrize("tx,ty", TYPES)
def test_strides_offsets_and_repeated_rows(tx, ty):
    """Views with padding between tokens and streams, streams apart from each
    other, bases off 16 bytes, coefficients as slices of one projection's
    output, and one row repeated over streams."""
    T, S, C = 11, 4, 96
    k = inputs(T, S, C, tx, ty)
    apart = dict(k)
    apart["x"] = torch.cat([k["x"].transpose(0, 1), rnd(90, S, 1, C, dtype=tx)], 1).contiguous()[:, :T].transpose(0, 1)
    apart["D"] = torch.cat([k["D"], rnd(91, T, S, 3, dtype=tx)], 2)[:, :, :C]
    wide = torch.cat([rnd(92, T, 1, dtype=ty), k["y"], rnd(93, T, 2, dtype=ty)], 1)
    apart["y"] = wide[:, 1:C + 1]
    apart["gate"] = torch.cat([k["gate"], k["gate"]], 1)[:, :C]
    slices = torch.cat([k["a"], k["b"], k["P"].reshape(T, S * S)], 1)
    apart["a"], apart["b"], apart["P"] = slices[:, :S], slices[:, S:2 * S], slices[:, 2 * S:].view(T, S, S)
    buf = torch.empty(C + 1, device=DEV)
    buf[1:] = k["w"]
    apart["w"] = buf[1:]
    assert not apart["x"].is_contiguous() and apart["w"].data_ptr() % 16 == 4
    everything(apart)
    one = dict(k)
    one["x"] = k["x"][:, :1].expand(T, S, C)
    one["gate"] = k["gate"][:1].expand(T, C)
    assert one["x"].stride(1) == 0 and one["gate"].stride(0) == 0
    everything(one)


def test_leading_dimensions_and_transposed_channels():
    x, y = rnd(1, 2, 3, 4, 40), rnd(2, 2, 3, 40)
    P, b = torch.softmax(rnd(3, 2, 3, 4, 4), -1), rnd(4, 2, 3, 4)
    out = block.leave(x, y, P, b)
    flat = block.leave(x.flatten(0, 1), y.flatten(0, 1), P.flatten(0, 1), b.flatten(0, 1))
    assert out.shape == x.shape and torch.equal(out.flatten(0, 1), flat)
    assert torch.equal(block.leave(x[0, 0], y[0, 0], P[0, 0], b[0, 0]), out[0, 0])
    turned = x.transpose(2, 3).contiguous().transpose(2, 3)
    assert turned.stride(3) != 1 and torch.equal(block.leave(turned, y, P.transpose(0, 1).contiguous().transpose(0, 1), b), out)
    # sequences cut from a longer buffer: the leading dimensions do not collapse
    assert torch.equal(block.enter(torch.cat([x, x], 1)[:, :3], b), block.enter(x, b))


def test_vector_and_element_paths_agree():
    """The same rows on and off 16-byte boundaries: only the order of the sums
    differs."""
    T, S, C = 37, 4, 512
    k = inputs(T, S, C, H, H)
    buf = torch.empty(T * S * C + 1, dtype=H, device=DEV)
    buf[1:] = k["x"].flatten()
    a = block.leave(k["x"], k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"])
    b = block.leave(buf[1:].view(T, S, C), k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"])
    # a row's rho may differ by a few 2^-24, which flips a bf16 rounding now and then
    assert (a != b).float().mean() < 1e-2 and (a.float() - b.float()).abs().max() <= 2.0 ** -6 * a.float().abs().max()


def test_plain_and_full_calls_agree(monkeypatch):
    """The extension module's short way and the Python code make the same calls."""
    class Nothing:
        def __getattr__(self, name):
            return lambda *args: None

    def results():
        got = []
        for S, tx, ty, coef, weight, act in ((4, H, H, F, F, "silu"), (1, F, H, F, H, None), (3, F, F, H, F, "linear")):
            for mix in (True, False):
                k = inputs(7, S, 88, tx, ty, act, mix, coef, weight)
                how = dict(gate=k["gate"], act=act or "sigmoid", weight=k["w"], norm=act != "linear", scale=0.25, eps=1e-5)
                nxt = dict(a_next=k["a"], weight_next=k["w2"], eps_next=1e-4)
                got.append(block.enter(k["x"], k["a"], k["w"], eps=1e-3, out_dtype=ty))
                got += block.enter_backward(k["dh"], k["x"], k["a"], k["w"], eps=1e-3, dres=k["D"])
                got += block.enter_backward(k["dh"], k["x"], k["a"], None)
                got.append(block.leave(k["x"], k["y"], k["P"], k["b"], **how))
                got += block.leave_enter(k["x"], k["y"], k["P"], k["b"], **how, **nxt)
                got += block.leave_backward(k["D"], k["x"], k["y"], k["P"], k["b"], **how)
                got += block.leave_enter_backward(k["D"], k["dh"], k["x"], k["x"], k["y"], k["P"], k["b"], **how, **nxt)
        return got

    plain = results()
    monkeypatch.setattr(block, "_module", Nothing())
    full = results()
    assert len(plain) == len(full)
    for p, q in zip(plain, full):
        assert (p is None) == (q is None)
        assert p is None or (p.dtype == q.dtype and torch.equal(p, q))


def test_no_tokens():
    x, y, w = torch.empty(0, 4, 64, device=DEV), torch.empty(0, 64, device=DEV), rnd(1, 64)
    assert block.enter(x, None, w).shape == (0, 64)
    out, h = block.leave_enter(x, y, weight=w, weight_next=w)
    assert out.shape == x.shape and h.shape == y.shape
    g = block.enter_backward(y, x, None, w)
    assert g.dx.shape == x.shape and torch.equal(g.dweight, torch.zeros_like(w))
    g = block.leave_backward(x, x, y, weight=w)
    assert torch.equal(g.dweight, torch.zeros_like(w)) and g.dy.shape == y.shape
    g = block.leave_enter_backward(x, y, x, x, y, weight=w, weight_next=w)
    assert torch.equal(g.dweight, torch.zeros_like(w)) and torch.equal(g.dweight_next, torch.zeros_like(w))


@pytest.mark.parametrize("C", [64, 65])
def test_rows_of_zeros(C):
    """A row of zeros has r = 1/sqrt(eps): finite results and gradients."""
    k = inputs(5, 4, C, F, F)
    k["x"][1], k["y"][1], k["x"][3], k["D"][3], k["dh"][3] = 0, 0, 0, 0, 0
    everything(k)
    k["P"][2], k["b"][2], k["a"][2] = 0, 0, 0  # coefficients that leave nothing
    everything(k)


@pytest.mark.parametrize("tx", [F, H])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
def test_what_is_not_finite_stays_in_its_token(tx, bad):
    """And, without a mixing matrix, in its stream."""
    T, S, C = 9, 4, 256
    k = inputs(T, S, C, tx, tx, act="silu")
    how = dict(gate=k["gate"], act="silu", weight=k["w"])
    clean = block.leave(k["x"], k["y"], k["P"], k["b"], **how)
    alone = block.leave(k["x"], k["y"], **how)
    x = k["x"].clone()
    x[4, 2, 17] = bad
    got = block.leave(x, k["y"], k["P"], k["b"], **how)
    rest = [t for t in range(T) if t != 4]
    assert torch.equal(got[rest], clean[rest]) and not torch.isfinite(got[4, :, 17]).any()
    keep = torch.ones(C, dtype=torch.bool, device=DEV)
    keep[17] = False
    assert torch.equal(got[4][:, keep], clean[4][:, keep])
    got = block.leave(x, k["y"], **how)
    same = torch.ones_like(alone, dtype=torch.bool)
    same[4, 2, 17] = False
    assert torch.equal(got[same], alone[same]) and not torch.isfinite(got[4, 2, 17])
    h = block.enter(x, k["a"], k["w"])
    assert torch.isfinite(h[rest]).all()
    g = block.leave_backward(k["D"], x, k["y"], k["P"], k["b"], **how)
    assert torch.isfinite(g.dx).all() and torch.isfinite(g.dy).all() and torch.isfinite(g.dP[rest]).all()
    assert not torch.isfinite(g.dP[4, :, 2]).any() and torch.isfinite(g.dP[4][:, [0, 1, 3]]).all()
    y = k["y"].clone()
    y[4, 17] = bad
    got = block.leave(k["x"], y, k["P"], k["b"], **how)
    assert torch.equal(got[rest], clean[rest])


def test_gates_far_out():
    """Saturated gates: sigmoid's tails and slopes neither overflow nor cancel."""
    g = torch.tensor([-1e4, -200.0, -89.0, -30.0, -1e-3, 0.0, 1e-3, 17.0, 30.0, 89.0, 200.0, 1e4], device=DEV)
    C = g.numel()
    y, x, D = torch.ones(1, C, device=DEV), torch.zeros(1, 1, C, device=DEV), torch.ones(1, 1, C, device=DEV)
    for act in ("sigmoid", "silu", "linear"):
        out = block.leave(x, y, gate=g[None], act=act, norm=False)
        d = block.leave_backward(D, x, y, gate=g[None], act=act, norm=False).dgate
        value, slope, mag = ob.gate_value(act, np64(g))
        # exp(-|g|) carries |g| 2^-24 of relative error from its argument; results below 2^-126 may be flushed
        lim = (16 + 3 * np.minimum(np.abs(np64(g)), 128)) * 2.0 ** -24
        assert (np.abs(np64(out)[0, 0] - value) <= lim * np.abs(value) + 2.0 ** -118).all()
        assert (np.abs(np64(d)[0] - slope) <= lim * mag + 2.0 ** -118).all()


def test_gradients_may_replace_their_inputs():
    T, S, C = 21, 4, 320
    k = inputs(T, S, C, H, H)
    want = block.enter_backward(k["dh"], k["x"], k["a"], k["w"], dres=k["D"])
    res = k["D"].clone()
    direct("hcb_enter_backward", dict(x=k["x"], dh=k["dh"], a=k["a"], w=k["w"], dres=res, dx=res), T, S, C, H)
    assert torch.equal(res, want.dx)


def test_every_gradient_alone():
    """Any subset of a backward pass's outputs gives what all of them give."""
    T, S, C = 19, 4, 136
    k = inputs(T, S, C, F, F)
    want = block.leave_backward(k["D"], k["x"], k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"])
    for field, name in (("dx", "dx"), ("dy", "dy"), ("dP", "dP"), ("db", "db"), ("dgate", "dgate"), ("dw", "dweight")):
        t = torch.full_like(getattr(want, name), 7.0)
        ws = torch.empty(block.workspace_bytes(T, C), dtype=torch.uint8, device=DEV) if field == "dw" else None
        direct("hcb_leave_backward", dict(dout=k["D"], x=k["x"], y=k["y"], P=k["P"], b=k["b"], gate=k["gate"], w=k["w"],
                                          workspace=ws, **{field: t}), T, S, C, F, act=1)
        assert torch.equal(t, getattr(want, name)), name


@pytest.mark.parametrize("T", [1, 500])
def test_results_repeat_bit_for_bit(T):
    k = inputs(T, 4, 1024, H, H)
    run = lambda: block.leave_enter_backward(k["D"], k["dh"], k["x"], k["x"], k["y"], k["P"], k["b"], gate=k["gate"],  # noqa: E731
                                             weight=k["w"], a_next=k["a"], weight_next=k["w2"])
    first = run()
    for _ in range(3):
        assert all(torch.equal(p, q) for p, q in zip(first, run()))


def test_autograd_matches_the_functions():
    T, S, C = 12, 4, 128
    k = inputs(T, S, C, F, F)
    leaf = {n: t.clone().requires_grad_() for n, t in k.items() if n not in ("D", "dh")}
    out, h = block.leave_enter(leaf["x"], leaf["y"], leaf["P"], leaf["b"], gate=leaf["gate"], act="silu", weight=leaf["w"],
                               a_next=leaf["a"], weight_next=leaf["w2"], scale=0.3)
    torch.autograd.backward([out, h], [k["D"], k["dh"]])
    g = block.leave_enter_backward(k["D"], k["dh"], out.detach(), k["x"], k["y"], k["P"], k["b"], gate=k["gate"], act="silu",
                                   weight=k["w"], a_next=k["a"], weight_next=k["w2"], scale=0.3)
    for n, d in zip(("x", "y", "P", "b", "gate", "w", "a", "w2"), g):
        assert torch.equal(leaf[n].grad, d), n
    for t in leaf.values():
        t.grad = None
    # the two halves one after the other: the same to fp32 rounding
    mid = block.leave(leaf["x"], leaf["y"], leaf["P"], leaf["b"], gate=leaf["gate"], act="silu", weight=leaf["w"], scale=0.3)
    h2 = block.enter(mid, leaf["a"], leaf["w2"])
    torch.autograd.backward([mid, h2], [k["D"], k["dh"]])
    for n, d in zip(("x", "y", "P", "b", "gate", "w", "a", "w2"), g):
        assert (leaf[n].grad - d).norm() <= 1e-5 * d.norm(), n


def test_autograd_of_one_repeated_row_and_unused_results():
    """Broadcast streams and gates: their gradients are summed over the copies."""
    T, S, C = 6, 4, 64
    e, gate = rnd(1, T, 1, C).requires_grad_(), rnd(2, C).requires_grad_()
    y, P = rnd(3, T, C), torch.softmax(rnd(4, T, S, S), -1)
    out, h = block.leave_enter(e.expand(T, S, C), y, P, gate=gate.expand(T, C))
    h.sum().backward()  # the gradient of `out` itself is zero
    x, g = e.detach().expand(T, S, C).contiguous(), gate.detach().expand(T, C).contiguous()
    d = block.leave_enter_backward(torch.zeros_like(x), torch.ones_like(y), out.detach(), x, y, P, gate=g)
    # sums of S and of T numbers in another order
    assert (e.grad - d.dx.sum(1, keepdim=True)).abs().max() <= 8 * 2.0 ** -23 * d.dx.abs().sum(1).max()
    assert (gate.grad - d.dgate.sum(0)).abs().max() <= 8 * 2.0 ** -23 * d.dgate.abs().sum(0).max()


def test_the_projection_and_the_block_together():
    """project -> enter -> leave, differentiated through the projection."""
    T, S, C = 8, 4, 32
    logits = rnd(1, T, S, S).requires_grad_()
    x, a, b, y, D = rnd(2, T, S, C), rnd(3, T, S), rnd(4, T, S), rnd(5, T, C), rnd(6, T, S, C)
    out = block.leave(x, y, b4.project(logits), b)
    out.backward(D)
    P = b4.project(logits.detach())
    dP = block.leave_backward(D, x, y, P, b).dP
    assert torch.equal(logits.grad, b4.backward(dP, P=P))


def test_other_streams_and_a_workspace():
    k = inputs(64, 4, 256, H, H)
    want = block.enter_backward(k["dh"], k["x"], k["a"], k["w"])
    ws = torch.empty(block.workspace_bytes(64, 256), dtype=torch.uint8, device=DEV)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        got = block.enter_backward(k["dh"], k["x"], k["a"], k["w"], workspace=ws)
    s.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(want, got))
    with pytest.raises(ValueError, match="workspace"):
        block.enter_backward(k["dh"], k["x"], k["a"], k["w"], workspace=ws[:-1])


def test_captured_in_a_graph():
    k = inputs(40, 4, 512, H, H)
    x = k["x"].clone()
    f = lambda: block.leave_enter(x, k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"], a_next=k["a"], weight_next=k["w2"])  # noqa: E731
    f()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out, h = f()
        d = block.leave_enter_backward(k["D"], k["dh"], out, x, k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"],
                                       a_next=k["a"], weight_next=k["w2"])
    x.copy_(rnd(77, 40, 4, 512, dtype=H))
    g.replay()
    torch.cuda.synchronize()
    want = f()
    assert torch.equal(out, want[0]) and torch.equal(h, want[1])
    again = block.leave_enter_backward(k["D"], k["dh"], out, x, k["y"], k["P"], k["b"], gate=k["gate"], weight=k["w"],
                                       a_next=k["a"], weight_next=k["w2"])
    assert all(torch.equal(p, q) for p, q in zip(d, again))


def test_offsets_past_32_bits():
    """A streams array of more than 2^31 elements: the last tokens (few tokens
    are summed by longer groups, so not bit for bit what a small array gives)."""
    T, S, C = 140000, 4, 4096
    x = torch.zeros(T, S, C, dtype=H, device=DEV)
    y = torch.zeros(T, C, dtype=H, device=DEV)
    tail = inputs(5, S, C, H, H)
    x[-5:], y[-5:] = tail["x"], tail["y"]
    assert x.numel() > 2 ** 31
    n = {k: np64(t) for k, t in tail.items()}
    out = block.leave(x, y, scale=0.5, weight=tail["w"])
    close(out[-5:], ob.leave(n["x"], n["y"], w=n["w"], scale=0.5)["out"])
    assert not out[:-5].any()
    del out
    h = block.enter(x, None, tail["w"])
    close(h[-5:], ob.enter(n["x"], None, n["w"])["h"])
    assert not h[:-5].any()
    del h
    d = torch.zeros_like(x)
    d[-5:] = tail["D"]
    g = block.leave_backward(d, x, y, b=torch.ones(T, S, device=DEV), weight=tail["w"])
    want = ob.leave_backward(n["D"], n["x"], n["y"], w=n["w"])
    close(g.dy[-5:], want["dy"])
    close(g.db[-5:], want["db"])
    assert not g.dy[:-5].any() and not g.db[:-5].any()


def test_refusals():
    x, y = rnd(1, 3, 4, 8), rnd(2, 3, 8)
    for f, text in ((lambda: block.leave(x, rnd(1, 3, 9)), "shape"), (lambda: block.leave(x, rnd(1, 4, 8)), "shape"),
                    (lambda: block.leave(x, y, rnd(1, 3, 4)), "shape"), (lambda: block.leave(x, y, b=rnd(1, 3, 5)), "shape"),
                    (lambda: block.leave(x, y, weight=rnd(1, 9)), "shape"), (lambda: block.leave(x, y, gate=y.bfloat16()), "gate"),
                    (lambda: block.leave(x, y, gate=y, act="relu"), "act"), (lambda: block.enter(rnd(1, 2, 9, 8)), "streams"),
                    (lambda: block.enter(x[..., :0]), "channels"), (lambda: block.enter(y[0]), "shape"),
                    (lambda: block.leave(x, y.cpu()), "CUDA"), (lambda: block.enter_backward(y, x, dres=x[:2]), "dres"),
                    (lambda: block.leave_backward(x.bfloat16(), x, y), "dout")):
        with pytest.raises(ValueError, match=text):
            f()
    for f in (lambda: block.enter(x.double()), lambda: block.leave(x.bfloat16(), y), lambda: block.enter(x, out_dtype=torch.half),
              lambda: block.enter(x.bfloat16(), out_dtype=F)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(b4.Birkhoff4Error, match="invalid"):
        block.enter(x, eps=-1.0)
