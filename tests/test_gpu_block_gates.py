"""Gates of fp32 rows far from zero: as exact as near it.

In units of 2^-24: e = exp(-|g|) is within 2 (one ulp), 1 + e adds 1, its
reciprocal 4 (two ulp), so 1 / (1 + e) is within 7 and e / (1 + e) within 10;
silu's value multiplies by g: 11.  Slopes: s (1 - s) is within 18, and
s (1 + g (1 - s)) within 10 + 12 + 1 of its magnitude s (1 + |g| (1 - s)).
"""
import numpy as np
import pytest
import torch

from birkhoff_projection_gb300 import block
from oracle import block as ob

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.mark.parametrize("act", ["sigmoid", "silu"])
@pytest.mark.parametrize("S,weight,C", [(1, True, 2048), (1, False, 2048), (2, True, 2001), (4, True, 4096), (3, False, 500)])
def test_fp32_gates_of_any_size(act, S, weight, C):
    """Each |gate| up to 80; y, weight and b are ones, there is no norm, x is zero."""
    T = 3
    g = (torch.rand(T, C, generator=torch.Generator().manual_seed(C)) * 160 - 80).to(DEV)
    x, y = torch.zeros(T, S, C, device=DEV), torch.ones(T, C, device=DEV)
    w = torch.ones(C, device=DEV) if weight else None
    b = torch.zeros(T, S, device=DEV)
    b[:, 0] = 1
    P = torch.eye(S, device=DEV).expand(T, S, S).contiguous() if S > 1 else None
    how = dict(gate=g, act=act, weight=w, norm=False)
    value, slope, mag = ob.gate_value(act, g.double().cpu().numpy())
    out = block.leave(x, y, P, b, **how)[:, 0].double().cpu().numpy()
    err = np.abs(out - value) / np.abs(value)
    assert err.max() <= 16 * 2.0 ** -24, err.max() * 2 ** 24
    D = torch.ones(T, S, C, device=DEV)
    grads = block.leave_backward(D, x, y, P, b, **how)
    for got, want, m, n in ((grads.dgate, slope, mag, 24), (grads.dy, value, np.abs(value), 16)):
        err = np.abs(got.double().cpu().numpy() - want) / m
        assert err.max() <= n * 2.0 ** -24, err.max() * 2 ** 24
