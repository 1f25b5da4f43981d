"""The largest tensor that an AdamW step takes, as adamw.h states it
(refusals: nothing is launched)."""
import ctypes
import os
import re

from birkhoff_projection_gb300 import _lib

FAKE = 0x10000  # never dereferenced


def test_a_tensor_beyond_the_limit_is_refused():
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    text = open(os.path.join(root, "include", "adamw.h")).read()
    most = 1 << int(re.search(r"#define ADAMW_MAX_ELEMENTS \(INT64_C\(1\) << (\d+)\)", text).group(1))
    o = _lib.AdamwOpts(p_dtype=_lib.B4_F32, g_dtype=_lib.B4_F32, state_bits=32, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8, step=1)
    for n in (most + 1, 2 ** 63 - 1, -1):
        t = (_lib.AdamwTensor * 2)(_lib.AdamwTensor(FAKE, FAKE, FAKE, FAKE, None, None, None, 4),
                                   _lib.AdamwTensor(FAKE, FAKE, FAKE, FAKE, None, None, None, n))
        assert _lib.lib().adamw_step(t, 2, ctypes.byref(o), None) == _lib.B4_EINVAL
