"""The block oracle's gradients against central differences of its forward
formulas, and its e4m3 rounding against the full table of e4m3 numbers."""
import numpy as np
import pytest

from oracle import block as ob

T, S, C = 2, 3, 5


def numbers(seed, *shape):
    return np.random.default_rng(seed).standard_normal(shape)


def differences(f, x, D, h=1e-6):
    """d/dx of sum(D f(x)), entry by entry."""
    got = np.zeros_like(x)
    for i in np.ndindex(x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        got[i] = ((f(up) - f(down)) * D).sum() / (2 * h)
    return got


def near(a, b):
    # central differences: truncation ~ h^2 and cancellation ~ 1e-16 / h, both about 1e-10 of values of order one
    assert np.abs(a - b).max() <= 1e-7 * max(1.0, np.abs(b).max())


@pytest.mark.parametrize("eps", [1e-6, 0.5])
def test_enter_gradients(eps):
    x, a, w, dh, res = numbers(1, T, S, C), numbers(2, T, S), numbers(3, C), numbers(4, T, C), numbers(5, T, S, C)
    g = ob.enter_backward(dh, x, a, w, eps, res)
    near(g["dx"][0] - res, differences(lambda t: ob.enter(t, a, w, eps)["h"][0], x, dh))
    near(g["da"][0], differences(lambda t: ob.enter(x, t, w, eps)["h"][0], a, dh))
    near(g["dweight"][0], differences(lambda t: ob.enter(x, a, t, eps)["h"][0], w, dh))


@pytest.mark.parametrize("act", [None, "sigmoid", "silu", "linear"])
@pytest.mark.parametrize("norm", [True, False])
@pytest.mark.parametrize("mix", [True, False])
def test_leave_gradients(act, norm, mix):
    x, y, w, D = numbers(1, T, S, C), numbers(2, T, C), numbers(3, C), numbers(4, T, S, C)
    P = numbers(5, T, S, S) if mix else None
    b = numbers(6, T, S)
    gate = None if act is None else numbers(7, T, C)

    def f(x=x, y=y, P=P, b=b, gate=gate, w=w):
        return ob.leave(x, y, P, b, gate, act, w, norm, 0.7, 1e-3)["out"][0]

    g = ob.leave_backward(D, x, y, P, b, gate, act, w, norm, 0.7, 1e-3)
    near(g["dx"][0], differences(lambda t: f(x=t), x, D))
    near(g["dy"][0], differences(lambda t: f(y=t), y, D))
    near(g["db"][0], differences(lambda t: f(b=t), b, D))
    near(g["dweight"][0], differences(lambda t: f(w=t), w, D))
    if mix:
        near(g["dP"][0], differences(lambda t: f(P=t), P, D))
    if gate is not None:
        near(g["dgate"][0], differences(lambda t: f(gate=t), gate, D))


def test_leave_enter_gradients():
    x, y, w, w2 = numbers(1, T, S, C), numbers(2, T, C), numbers(3, C), numbers(4, C)
    P, b, a2 = numbers(5, T, S, S), numbers(6, T, S), numbers(7, T, S)
    D, dh = numbers(8, T, S, C), numbers(9, T, C)

    def loss(**new):
        k = dict(x=x, y=y, P=P, b=b, w=w, a2=a2, w2=w2) | new
        out = ob.leave(k["x"], k["y"], k["P"], k["b"], w=k["w"])["out"][0]
        return (out * D).sum() + (ob.enter(out, k["a2"], k["w2"])["h"][0] * dh).sum()

    out = ob.leave(x, y, P, b, w=w)["out"][0]
    g = ob.leave_enter_backward(D, dh, out, x, y, P, b, w=w, a_next=a2, w_next=w2)
    for name, key, t in (("dx", "x", x), ("dy", "y", y), ("dP", "P", P), ("db", "b", b), ("dweight", "w", w),
                         ("da_next", "a2", a2), ("dweight_next", "w2", w2)):
        near(g[name][0], differences(lambda v: np.array(loss(**{key: v})), t, 1.0))


def test_e4m3_rounds_to_the_nearest_number():
    table = np.array([(m / 8 if e == 0 else 1 + m / 8) * 2.0 ** (max(e, 1) - 7)
                      for e in range(16) for m in range(8)][:-1])
    assert table[-1] == ob.TOP and table[1] == ob.LEAST
    assert (ob.e4m3(table) == table).all() and (ob.e4m3(-table) == -table).all()
    mid = (table[1:] + table[:-1]) / 2
    even = np.where(np.arange(len(mid)) % 2 == 0, table[:-1], table[1:])
    assert (ob.e4m3(mid) == even).all()
    assert (ob.e4m3(mid * (1 + 1e-7)) == table[1:]).all()
    assert (ob.e4m3(mid * (1 - 1e-7)) == table[:-1]).all()


def test_eight_bit_blocks_hold_their_values_to_half_a_step():
    x = (numbers(1, 1000) * np.exp(numbers(2, 1000))).astype(np.float32)
    for root in (False, True):
        v = np.abs(x) if root else x
        code, scale = ob.encode(v, root)
        back = ob.decode(code, scale)
        most = np.repeat(np.abs(np.pad(v, (0, 24))).reshape(-1, 128).max(1), 128)[:1000]
        # half a step: 2^-4 of the value, or half of 2^-9 / 448 of the largest below the normal numbers
        # (a positive root is never rounded to zero: a whole step); three fp32 roundings of 2^-24 beside
        small = (2.0 ** -9 if root else 2.0 ** -10) / 448 * most
        assert (np.abs(back - v) <= np.maximum(np.abs(v) * (2.0 ** -4 + 1e-6), small)).all()
        if root:
            assert (back[v > 0] > 0).all()
