"""Calls of the block operators from Python: what they take, what they
allocate and what they raise."""
import gc

import pytest
import torch

from birkhoff_projection_gb300 import _lib, block, optim

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_out_of_memory_is_torchs_own_error():
    """From the extension module as from torch: what a caller catches to retry with less."""
    gc.collect()
    torch.cuda.empty_cache()  # so that these have segments of their own, with no room beside them
    x = torch.zeros(1 << 14, 4, 2048, device=DEV)  # 512 MB, its row 128
    dh = torch.zeros(1 << 14, 2048, device=DEV)
    torch.cuda.synchronize()
    torch.cuda.empty_cache()
    torch.cuda.set_per_process_memory_fraction(1e-6)
    try:
        for call in (lambda: block.enter(x), lambda: block.leave(x, dh), lambda: block.enter_backward(dh, x),
                     lambda: block.leave_backward(x, x, dh)):
            with pytest.raises(torch.OutOfMemoryError):
                call()
    finally:
        torch.cuda.set_per_process_memory_fraction(1.0)
    assert block.enter(x).shape == dh.shape


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_last_token_of_a_long_buffer(dtype):
    """Tokens that are further apart than the library's strides go (2^29)."""
    L, S, C = 33000, 4, 4096
    buf = torch.empty(2, L, S, C, dtype=dtype, device=DEV)
    rows = torch.empty(2, 1 << 29, dtype=dtype, device=DEV)[:, None, :C]
    assert buf.stride(0) > 1 << 29 and rows.stride(0) == 1 << 29
    g = torch.Generator().manual_seed(0)
    buf[:, -1] = torch.randn(2, S, C, generator=g).to(dtype).to(DEV)
    rows.copy_(torch.randn(2, 1, C, generator=g))
    x, packed, y = buf[:, -1:], buf[:, -1:].contiguous(), rows.contiguous()
    assert torch.equal(block.enter(x), block.enter(packed))
    assert torch.equal(block.leave(x, rows, gate=rows), block.leave(packed, y, gate=y))
    for p, q in ((block.enter_backward(rows, x, dres=x), block.enter_backward(y, packed, dres=packed)),
                 (block.leave_enter_backward(x, rows, x, x, rows), block.leave_enter_backward(packed, y, packed, packed, y))):
        assert all(s is None and t is None or torch.equal(s, t) for s, t in zip(p, q))


def test_without_the_extension_module(monkeypatch):
    """Where it cannot be built, the same results come through the Python code."""
    def results():
        torch.manual_seed(0)
        x, y = torch.randn(5, 4, 72, device=DEV), torch.randn(5, 72, device=DEV)
        w = torch.nn.Parameter(torch.randn(72, device=DEV))
        opt = optim.AdamW([w], state_bits=8)
        out, h = block.leave_enter(x, y, weight=w, weight_next=w)
        (out.sum() + (h * y).sum()).backward()
        opt.step()
        return out.detach(), h.detach(), w.grad, w.detach()

    want = results()
    monkeypatch.setattr(_lib, "_binding", _lib._NoBinding())
    monkeypatch.setattr(block, "_module", None)
    assert all(torch.equal(p, q) for p, q in zip(want, results()))
