"""float64 oracle of the hyper-connection block operators and of the AdamW
step (numpy; test infrastructure).

Every result of the block operators comes with a magnitude: the same
expression with its terms' absolute values, so that an fp32 evaluation of n
roundings is within about n 2^-24 magnitude of the value whatever cancels in
it.  The formulas are those of include/hc_block.h and include/adamw.h, pinned
to finite differences in tests/test_oracle_block.py.
"""
from __future__ import annotations

import numpy as np


def _ones(a, shape):
    return np.ones(shape) if a is None else np.asarray(a, np.float64)


def gate_value(act, g):
    """(act(g), act'(g), magnitude of act'(g))."""
    g = np.asarray(g, np.float64)
    if act == "linear":
        return g, np.ones_like(g), np.ones_like(g)
    with np.errstate(over="ignore"):
        s = 1 / (1 + np.exp(-g))
        rest = 1 / (1 + np.exp(g))
    if act == "sigmoid":
        return s, s * rest, s * rest
    return g * s, s * (1 + g * rest), s * (1 + np.abs(g) * rest)


def _aggregate(x, a, eps):
    """u, its magnitude, r, and the factor by which u's cancellation enters r."""
    u = np.einsum("ts,tsc->tc", a, x)
    um = np.einsum("ts,tsc->tc", np.abs(a), np.abs(x))
    ms = (u * u).mean(1, keepdims=True) + eps
    with np.errstate(divide="ignore", invalid="ignore"):
        return u, um, 1 / np.sqrt(ms), (np.abs(u) * um).mean(1, keepdims=True) / ms


def enter(x, a=None, w=None, eps=1e-6):
    x = np.asarray(x, np.float64)
    T, S, C = x.shape
    a, w = _ones(a, (T, S)), _ones(w, C)
    u, um, r, q = _aggregate(x, a, eps)
    return {"h": (w * u * r, np.abs(w) * r * (um + np.abs(u) * q))}


def enter_backward(dh, x, a=None, w=None, eps=1e-6, dres=None):
    x, dh = np.asarray(x, np.float64), np.asarray(dh, np.float64)
    T, S, C = x.shape
    a, w = _ones(a, (T, S)), _ones(w, C)
    u, um, r, q = _aggregate(x, a, eps)
    G = w * dh
    k = (G * u).mean(1, keepdims=True) * r * r
    km = (np.abs(G) * um).mean(1, keepdims=True) * r * r
    du = r * (G - k * u)
    dum = r * (np.abs(G) + km * um) * (1 + q)
    res = 0.0 if dres is None else np.asarray(dres, np.float64)
    return {
        "dx": (a[:, :, None] * du[:, None] + res, np.abs(a)[:, :, None] * dum[:, None] + np.abs(res)),
        "da": (np.einsum("tc,tsc->ts", du, x), np.einsum("tc,tsc->ts", dum, np.abs(x))),
        "dweight": ((dh * u * r).sum(0), (np.abs(dh) * um * r * (1 + q)).sum(0)),
    }


def _value(y, gate, act, w, norm, scale, eps):
    """z, act, slope (and its magnitude), rho."""
    rho = 1 / np.sqrt((y * y).mean(1, keepdims=True) + eps) if norm else np.ones((y.shape[0], 1))
    q, slope, slm = (1.0, 0.0, 0.0) if gate is None else gate_value(act, gate)
    return y * rho * w, q, slope, slm, rho


def leave(x, y, P=None, b=None, gate=None, act="sigmoid", w=None, norm=True, scale=1.0, eps=1e-6):
    x, y = np.asarray(x, np.float64), np.asarray(y, np.float64)
    T, S, C = x.shape
    b, w = _ones(b, (T, S)), _ones(w, C)
    z, q, *_ = _value(y, gate, act, w, norm, scale, eps)
    v = scale * q * z
    if P is None:
        mixed, mm = x, np.abs(x)
    else:
        P = np.asarray(P, np.float64)
        mixed, mm = np.einsum("tij,tjc->tic", P, x), np.einsum("tij,tjc->tic", np.abs(P), np.abs(x))
    return {"out": (mixed + b[:, :, None] * v[:, None], mm + np.abs(b)[:, :, None] * np.abs(v)[:, None])}


def leave_backward(D, x, y, P=None, b=None, gate=None, act="sigmoid", w=None, norm=True, scale=1.0, eps=1e-6, Dm=None):
    """Dm: the magnitude of D (its own absolute value unless given)."""
    D, x, y = (np.asarray(t, np.float64) for t in (D, x, y))
    Dm = np.abs(D) if Dm is None else Dm
    T, S, C = x.shape
    b, w = _ones(b, (T, S)), _ones(w, C)
    z, q, slope, slm, rho = _value(y, gate, act, w, norm, scale, eps)
    v = scale * q * z
    got = {}
    if P is None:
        got["dx"] = (D, Dm)
    else:
        P = np.asarray(P, np.float64)
        got["dx"] = (np.einsum("tij,tic->tjc", P, D), np.einsum("tij,tic->tjc", np.abs(P), Dm))
        got["dP"] = (np.einsum("tic,tjc->tij", D, x), np.einsum("tic,tjc->tij", Dm, np.abs(x)))
    got["db"] = (np.einsum("tic,tc->ti", D, v), np.einsum("tic,tc->ti", Dm, np.abs(v)))
    dv, dvm = np.einsum("ti,tic->tc", b, D), np.einsum("ti,tic->tc", np.abs(b), Dm)
    if gate is not None:
        got["dgate"] = (scale * dv * slope * z, abs(scale) * dvm * slm * np.abs(z))
    dz, dzm = scale * q * dv, np.abs(scale * q) * dvm
    g, gm = dz * w, dzm * np.abs(w)
    if norm:
        k, km = (g * y).mean(1, keepdims=True) * rho ** 2, (gm * np.abs(y)).mean(1, keepdims=True) * rho ** 2
    else:
        k = km = 0.0
    got["dy"] = (rho * (g - k * y), rho * (gm + km * np.abs(y)))
    got["dweight"] = ((dz * y * rho).sum(0), (dzm * np.abs(y) * rho).sum(0))
    return got


def leave_enter_backward(dout, dh, out, x, y, P=None, b=None, gate=None, act="sigmoid", w=None, norm=True, scale=1.0,
                         eps=1e-6, a_next=None, w_next=None, eps_next=1e-6):
    """The gradient is not rounded between the two halves."""
    e = enter_backward(dh, out, a_next, w_next, eps_next, dout)
    got = leave_backward(e["dx"][0], x, y, P, b, gate, act, w, norm, scale, eps, e["dx"][1])
    got["da_next"], got["dweight_next"] = e["da"], e["dweight"]
    return got


# ---------------------------------------------------------------------------
# AdamW
# ---------------------------------------------------------------------------
BLOCK, TOP, LEAST = 128, 448.0, 2.0 ** -9


def e4m3(q):
    """The nearest e4m3 number to float32 q, |q| <= 448 (ties to even; steps
    of 2^-9 below 2^-6); NaN stays."""
    q = np.asarray(q, np.float64)
    _, e = np.frexp(np.maximum(np.abs(q), 2.0 ** -6))
    step = np.ldexp(1.0, e - 4)
    return np.round(q / step) * step


def encode(x, root):
    """(e4m3 values, scales) of float32 x, blocks of 128, in the library's
    fp32 arithmetic."""
    x = np.asarray(x, np.float32)
    n = x.size
    pad = np.zeros(-(-n // BLOCK) * BLOCK, np.float32)
    pad[:n] = x
    blocks = pad.reshape(-1, BLOCK)
    mag = np.where(np.isfinite(blocks), np.abs(blocks), np.float32(0))
    most = mag.max(1)
    with np.errstate(divide="ignore", over="ignore", invalid="ignore"):
        inv = np.where(most > 0, np.minimum(np.float32(TOP) * (np.float32(1) / most), np.float32(3.0e38)), np.float32(0)).astype(np.float32)
        q = blocks * inv[:, None]
        if root:
            q = np.where(blocks > 0, np.maximum(q, np.float32(LEAST)), q)
        q = np.where(np.isfinite(blocks), q, np.float32(np.nan))
    code = np.minimum(np.maximum(e4m3(q), -TOP), TOP)
    return code.reshape(-1)[:n], most * (np.float32(1) / np.float32(TOP))


def decode(code, scale):
    """float32 values of e4m3 numbers and their scales."""
    code = np.asarray(code, np.float32)
    return code * np.repeat(np.asarray(scale, np.float32), BLOCK)[:code.size]


def adamw_moments(g, m, v, beta1, beta2, grad_scale=None):
    """The new moments in float32, every product and sum rounded by itself:
    what the library computes, bit for bit."""
    f = np.float32
    g, m, v = (np.asarray(t, f) for t in (g, m, v))
    with np.errstate(over="ignore", invalid="ignore"):
        if grad_scale is not None:
            g = g * f(grad_scale)
        m = f(beta1) * m + f(1.0 - beta1) * g
        v = f(beta2) * v + f(1.0 - beta2) * (g * g)
    return m, v


def adamw_weights(p, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """(new weights, size of the update) in float64 from the new moments."""
    p, m, v = (np.asarray(t, np.float64) for t in (p, m, v))
    with np.errstate(over="ignore", invalid="ignore", divide="ignore"):
        up = lr / (1 - beta1 ** step) * m / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    return p * (1 - lr * weight_decay) - up, np.abs(up)
