"""Many tokens to a group of threads: the kernels' loops over tokens go round
several times (a group takes 1 to 4 tokens at a time, and a GPU holds up to
some 2500 groups of a warp or 300 of a long row), so that rows copied ahead,
slots used again, sums in their other buffer and a last, partial round are all
compared with the oracle.  One stream without a mixing matrix, whose kernels
keep a row in registers, is tested over its types and limits.

Tolerance: as for the other tests of these operators, 256 2^-24 of a value's
magnitude: a weight gradient's longest chain of additions is 30001 / 2400
tokens of a group, 8 groups of a CTA, 20 rows of CTAs in a thread and 32
threads, 73 in all.
"""
import pytest
import torch

from birkhoff_projection_gb300 import block
from oracle import block as ob
from test_gpu_block import F, H, TYPES, compare, everything, inputs, np64, rnd

pytestmark = pytest.mark.gpu


def one_stream(T, C, tx, ty, act, coef, weight, seed=0):
    """No P; coef: the coefficients' type, None for none of them."""
    k = inputs(T, 1, C, tx, ty, act, True, coef or F, weight, seed)
    k["P"] = None
    if coef is None:
        k["a"] = k["b"] = None
    return k


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("act", [None, "silu"])
@pytest.mark.parametrize("T,C,coef", [(1, 1, F), (3, 7, None), (1, 4096, H), (3, 2048, F), (30001, 256, F), (1403, 4096, None),
                                      (1403, 2048, F), (2003, 1001, H), (1403, 4095, None), (1203, 4097, F), (901, 8192, None)])
def test_one_stream(T, C, coef, act, tx, ty):
    everything(one_stream(T, C, tx, ty, act, coef, F), act or "sigmoid")


@pytest.mark.parametrize("tx,ty", TYPES)
@pytest.mark.parametrize("weight", [F, H])
@pytest.mark.parametrize("C,coef", [(264, H), (2048, F), (265, F)])
def test_one_stream_types_of_weights(C, coef, weight, tx, ty):
    everything(one_stream(1500, C, tx, ty, "linear", coef, weight), "linear", norm=False, scale=-1.25)


@pytest.mark.parametrize("tx,ty", TYPES)
def test_one_stream_off_16_bytes(tx, ty):
    """Bases of one element behind a 16-byte boundary."""
    T, C = 1403, 2048
    k = one_stream(T, C, tx, ty, "sigmoid", F, F)
    for name in ("x", "y", "gate", "D", "dh"):
        buf = torch.empty(k[name].numel() + 1, dtype=k[name].dtype, device=k[name].device)
        buf[1:] = k[name].flatten()
        k[name] = buf[1:].view(k[name].shape)
    everything(k)


@pytest.mark.parametrize("tx,ty,sizes", [(tx, ty, s) for tx, ty in TYPES for s in (
    (5001, 4, 64), (5001, 2, 64), (5001, 4, 33), (5001, 8, 24), (1001, 2, 2048))] + [(H, H, (1001, 4, 5120)), (F, F, (1001, 3, 2000))])
def test_several_streams(tx, ty, sizes):
    everything(inputs(*sizes, tx, ty, seed=1))


def test_without_a_weight():
    """Several streams and one: the kernels that check everything at run time."""
    for S in (1, 4):
        k = inputs(5001, S, 96, H, H, seed=2)
        k["w"] = k["w2"] = None
        if S == 1:
            k["P"] = None
        everything(k)


@pytest.mark.parametrize("gate", [True, False])
def test_a_row_of_zeros_in_every_place_of_a_round(gate):
    """One stream: tokens whose y and streams are zero among others (a row's
    factor is then 1 / sqrt(eps), in this token alone)."""
    T, C = 1400, 4096
    k = one_stream(T, C, H, H, "silu" if gate else None, F, F)
    zero = torch.arange(T, device=k["x"].device) % 7 < 2
    k["x"][zero], k["y"][zero], k["D"][zero], k["dh"][zero] = 0, 0, 0, 0
    everything(k, "silu" if gate else "sigmoid", eps=1e-3, eps2=1e-3)


def test_one_stream_past_32_bits():
    """Rows beyond 2^31 elements."""
    T, C = 600001, 4096
    x = torch.zeros(T, 1, C, dtype=H, device="cuda:0")
    y, n = x[:, 0], 5
    tail = one_stream(n, C, H, H, None, None, F)
    x[-n:] = tail["x"]
    assert x.numel() > 2 ** 31
    t = {name: np64(v) for name, v in tail.items()}
    own = t["x"][:, 0]
    out, h = block.leave_enter(x, y, weight=tail["w"], weight_next=tail["w2"])
    from test_gpu_block import close
    close(out[-n:], ob.leave(t["x"], own, w=t["w"])["out"])
    assert not out[:-n].any() and not h[:-n].any()
    d = torch.zeros_like(x)
    d[-n:] = tail["D"]
    g = block.leave_enter_backward(d, y, out, x, y, weight=tail["w"], weight_next=tail["w2"])
    want = ob.leave_enter_backward(t["D"], own, np64(out[-n:]), t["x"], own, w=t["w"], w_next=t["w2"])
    close(g.dx[-n:], want["dx"])
    close(g.dy[-n:], want["dy"])
    assert not g.dx[:-n].any() and not g.dy[:-n].any()
