"""What block.py hands to the library for tensors of any strides (meta tensors:
no memory, no GPU)."""
import pytest
import torch

from birkhoff_projection_gb300 import block

MOST = 2 ** 29 - 1  # the largest stride that the library takes


def far(shape, strides, dtype=torch.float32):
    return torch.empty_strided(shape, strides, dtype=dtype, device="meta")


@pytest.mark.parametrize("strides,kept", [((MOST, 64, 1), True), ((64, MOST, 1), True), ((MOST + 1, 64, 1), False),
                                          ((64, MOST + 1, 1), False), ((2 ** 33, 2 ** 32, 1), False), ((0, 0, 1), True),
                                          ((512, 64, 2), False)])
def test_streams(strides, kept):
    t = far((3, 2, 64), strides)
    got, _, ts, ss = block._streams(t, "x", t.shape, t.dtype, t.get_device())
    assert (ts, ss) == (strides[:2] if kept else (128, 64)) == got.stride()[:2]
    t = far((2, 1, 2, 64), (strides[0], 1 << 40, *strides[1:]))  # the last token of two long sequences
    got, _, ts, ss = block._streams(t, "x", t.shape, t.dtype, t.get_device())
    assert (ts, ss) == (strides[:2] if kept else (128, 64))


@pytest.mark.parametrize("stride,kept", [(MOST, True), (MOST + 1, False), (2 ** 40, False)])
def test_rows_and_coefficients(stride, kept):
    t = far((3, 64), (stride, 1))
    assert block._row(t, "y", t.shape, t.dtype, t.get_device())[2] == (stride if kept else 64)
    t = far((3, 4), (stride, 1))
    assert block._few(t, "a", t.shape, 1, t.get_device())[3] == (stride if kept else 4)
    t = far((3, 4, 4), (stride, 4, 1))
    assert block._few(t, "P", t.shape, 2, t.get_device())[3] == (stride if kept else 16)


def test_one_token_whose_stride_means_nothing():
    t = far((1, 2, 64), (2 ** 40, 128, 1))
    assert block._streams(t, "x", t.shape, t.dtype, t.get_device())[2] <= MOST
