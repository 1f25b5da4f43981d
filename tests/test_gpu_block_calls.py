"""Calls of the block operators from Python: what they take, what they
allocate and what they raise."""
import pytest
import torch

from birkhoff_projection_gb300 import block

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def test_out_of_memory_is_torchs_own_error():
    """From the extension module as from torch: what a caller catches to retry with less."""
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
