"""Gradients through a sum of streams that nearly cancels.

Two streams alike to 1/1000 and coefficients of 1 and about -1 + 1/1000: u is
a thousandth of the streams.  It is exact up to one rounding (1 x is exact, and
the second product is fused), so every result is held to a magnitude in which
the streams enter through |u|, not through the sum of |a_s x_s|: what a sum
over u itself reaches, and one over the streams' sums <u, x_s> does not.

Tolerance: N 2^-24 of the magnitude and half a step of the type.  N = 256: a
sum over a row is at most 64 additions in a thread (16384 channels in a group
of 128 threads of pairs), 5 in a warp and 16 over warps, a weight gradient's
at most 40 over tokens and CTAs, and a result multiplies up to three of them;
as a norm 16, the root of it.
"""
import numpy as np
import pytest
import torch

from birkhoff_projection_gb300 import block
from oracle.block import gate_value

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
F, H = torch.float32, torch.bfloat16
N = 256


def np64(t):
    return t.detach().double().cpu().numpy()


def close(got, value, mag, name):
    half = torch.finfo(got.dtype).eps / 2
    err = np.abs(np64(got) - value)
    lim = N * 2.0 ** -24 * mag + half * np.abs(value) + 1e-37
    assert (err <= lim).all(), "%s: %g of the limit" % (name, (err / lim).max())
    norm = np.linalg.norm
    assert norm(err) <= 16 * 2.0 ** -24 * norm(mag) + half * norm(value) + 1e-37, name


def gradients(dh, x, a, w, eps):
    """dx, da and dw of enter with their magnitudes, in 64 bits."""
    u = np.einsum("ts,tsc->tc", a, x)
    r = 1 / np.sqrt((u * u).mean(1, keepdims=True) + eps)
    G = w * dh
    k, km = (G * u).mean(1, keepdims=True) * r * r, np.abs(G * u).mean(1, keepdims=True) * r * r
    du, dum = r * (G - k * u), r * (np.abs(G) + km * np.abs(u))
    return {"dx": (a[:, :, None] * du[:, None], np.abs(a)[:, :, None] * dum[:, None]),
            "da": (np.einsum("tc,tsc->ts", du, x), np.einsum("tc,tsc->ts", dum, np.abs(x))),
            "dw": ((dh * u * r).sum(0), np.abs(dh * u * r).sum(0))}


def make(T, S, C, tx, ty, along):
    g = torch.Generator().manual_seed(T + S + C)
    x = torch.zeros(T, S, C)
    x[:, 0] = torch.randn(T, C, generator=g)
    x[:, -1] = x[:, 0] * (1 + torch.randn(T, C, generator=g) / 1000)  # alike, but their sums <u, x_s> round apart
    a = torch.zeros(T, S)
    a[:, 0], a[:, -1] = 1.0, -1.0 + torch.rand(T, generator=g) / 500
    w = 1 + 0.2 * torch.randn(C, generator=g)
    dh = torch.randn(T, C, generator=g)
    if along:  # a gradient along the streams, whose share along u the norm takes out again
        dh = dh / 16 + x[:, 0]
    return x.to(tx).to(DEV), a.to(DEV), w.to(DEV), dh.to(ty).to(DEV)


SIZES = [(40, 2, 4096), (40, 4, 4096), (9, 3, 512), (9, 8, 640), (33, 4, 1001), (5, 2, 16384), (5, 4, 16384), (5, 5, 1000)]


@pytest.mark.parametrize("tx,ty", [(F, F), (H, H), (F, H)])
@pytest.mark.parametrize("along", [False, True])
@pytest.mark.parametrize("T,S,C", SIZES)
def test_enter(T, S, C, tx, ty, along):
    x, a, w, dh = make(T, S, C, tx, ty, along)
    got = block.enter_backward(dh, x, a, w, eps=1e-12)
    want = gradients(np64(dh), np64(x), np64(a), np64(w), 1e-12)
    for name, t in (("dx", got.dx), ("da", got.da), ("dw", got.dweight)):
        close(t, *want[name], name)


@pytest.mark.parametrize("tx,ty", [(F, F), (H, H), (F, H)])
@pytest.mark.parametrize("along", [False, True])
@pytest.mark.parametrize("T,S,C", SIZES)
@pytest.mark.parametrize("mix", [True, False])
def test_leave_enter(mix, T, S, C, tx, ty, along):
    """The same of the next block's input: with no other gradient, and with
    the identity for P."""
    out, a, w, dh = make(T, S, C, tx, ty, along)
    y = torch.randn(T, C, generator=torch.Generator().manual_seed(1)).to(ty).to(DEV)
    P = torch.eye(S, device=DEV).expand(T, S, S) if mix else None
    got = block.leave_enter_backward(torch.zeros_like(out), dh, out, out, y, P, weight=w, a_next=a, weight_next=w,
                                     eps_next=1e-12)
    want = gradients(np64(dh), np64(out), np64(a), np64(w), 1e-12)
    for name, t in (("dx", got.dx), ("da", got.da_next), ("dw", got.dweight_next)):
        close(t, *want[name], name)


@pytest.mark.parametrize("tx,ty", [(F, F), (H, H), (F, H)])
@pytest.mark.parametrize("along", [False, True])
@pytest.mark.parametrize("T,S,C", SIZES)
@pytest.mark.parametrize("act,mix,enters", [(None, True, False), ("sigmoid", True, False), (None, False, False), ("silu", True, True)])
def test_leave(act, mix, enters, T, S, C, tx, ty, along):
    """The streams' gradients nearly cancel in dv = sum_i b_i D_i, of which
    <w act dv, y> is a sum: dy.  along: y is along dv, the norm takes that share out."""
    D, b, w, y = make(T, S, C, tx, ty, along)
    g = torch.Generator().manual_seed(2)
    x = torch.randn(T, S, C, generator=g).to(tx).to(DEV)
    gate = None if act is None else torch.randn(T, C, generator=g).to(ty).to(DEV)
    P = torch.eye(S, device=DEV).expand(T, S, S) if mix else None
    how = dict(gate=gate, act=act or "sigmoid", weight=w, scale=0.5, eps=1e-12)
    if enters:  # and with no gradient through the next block's input
        got = block.leave_enter_backward(D, torch.zeros_like(y), x, x, y, P, b, weight_next=w, **how)
    else:
        got = block.leave_backward(D, x, y, P, b, **how)
    d, n, q, slope = np64(D), np64(y), 1.0, None
    dv = np.einsum("ts,tsc->tc", np64(b), d)
    rho = 1 / np.sqrt((n * n).mean(1, keepdims=True) + 1e-12)
    if act is not None:
        q, slope, slm = gate_value(act, np64(gate))
        z = n * rho * np64(w)
        close(got.dgate, 0.5 * dv * slope * z, 0.5 * np.abs(dv * z) * slm, "dgate")
    G = 0.5 * q * dv * np64(w)
    k, km = (G * n).mean(1, keepdims=True) * rho ** 2, np.abs(G * n).mean(1, keepdims=True) * rho ** 2
    close(got.dy, rho * (G - k * n), rho * (np.abs(G) + km * np.abs(n)), "dy")
    dz = 0.5 * q * dv * n * rho
    close(got.dweight, dz.sum(0), np.abs(dz).sum(0), "dweight")
