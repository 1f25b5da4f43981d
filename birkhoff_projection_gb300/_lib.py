"""ctypes loader for libbirkhoff4.so (the C ABI of include/birkhoff4.h).

Only argument marshalling lives here.  If the library cannot be built or
loaded, every call raises: there is no fallback path.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

from . import _build

_lock = threading.Lock()
_lib = None

B4_OK, B4_EINVAL, B4_ECUDA, B4_ENOTIMPL, B4_ESCRATCH = 0, 1, 2, 3, 4
B4_F32, B4_BF16 = 0, 1
B4_SCHED_DEFAULT, B4_SCHED_QUEUE, B4_SCHED_LANE, B4_SCHED_LANES4 = 0, 1, 2, 3

# Every function the header declares, with its ctypes signature.
_vp = ctypes.c_void_p
_i64 = ctypes.c_int64
_int = ctypes.c_int
SIGNATURES = {
    "birkhoff4_forward": (_int, [_vp, _vp, _vp, _i64, _vp]),
    "birkhoff4_forward_bf16": (_int, [_vp, _vp, _vp, _i64, _vp]),
    "birkhoff4_forward_ex": (_int, [_vp, _vp, _vp, _i64, _vp, _vp]),
    "birkhoff4_backward": (_int, [_vp, _vp, _vp, _vp, _i64, _vp]),
    "birkhoff4_backward_bf16": (_int, [_vp, _vp, _vp, _vp, _i64, _vp]),
    "birkhoff4_forward_backward": (_int, [_vp, _vp, _vp, _vp, _i64, _vp]),
    "birkhoff4_forward_backward_bf16": (_int, [_vp, _vp, _vp, _vp, _i64, _vp]),
    "birkhoff4_forward_backward_ex": (_int, [_vp, _vp, _vp, _vp, _i64, _vp, _vp]),
    "birkhoff4_forward_backward_host": (_int, [_vp, _vp, _vp, _vp, _i64, ctypes.c_int32, _vp,
                                               ctypes.c_size_t, _vp, ctypes.c_int32]),
    "birkhoff4_forward_backward_host_static": (_int, [_vp, _vp, _vp, _vp, _i64, ctypes.c_int32,
                                                      _i64, _vp, ctypes.c_int32]),
    "birkhoff4_forward_nxn": (_int, [_vp, _vp, _vp, ctypes.c_int32, _i64, _vp]),
    "birkhoff4_forward_backward_mapped": (_int, [_vp, _vp, _vp, _vp, _i64, ctypes.c_int32, _vp]),
    "eot_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, ctypes.c_int32, ctypes.c_int32]),
    "eot_update": (_int, [_vp, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_int32, ctypes.c_float,
                          ctypes.c_int32, _vp, ctypes.c_size_t, _vp]),
    "eot_transport_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, ctypes.c_int32]),
    "eot_transport": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64,
                             ctypes.c_int32, ctypes.c_float, _vp, ctypes.c_size_t, _vp]),
    "eot_apply_plan_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, ctypes.c_int32, ctypes.c_int32]),
    "eot_apply_plan": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, ctypes.c_int32, _vp, _vp, _i64,
                              _i64, ctypes.c_int32, ctypes.c_float, _vp, ctypes.c_size_t, _vp]),
    "eot_transport_schedule": (_int, [_i64, ctypes.c_int32, ctypes.c_int32, _vp]),
    "eot_hvp_workspace_bytes": (ctypes.c_size_t, [_i64, _i64, ctypes.c_int32]),
    "eot_hvp": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_int32,
                       ctypes.c_float, ctypes.c_int32, _vp, ctypes.c_size_t, _vp]),
    "eot_sinkhorn": (_int, [_vp, _vp, _vp, _vp, _vp, _vp, _i64, _i64, ctypes.c_int32,
                            ctypes.c_float, ctypes.c_int32, ctypes.c_int32, _vp, ctypes.c_size_t,
                            _vp]),
    "birkhoff4_backward_nxn": (_int, [_vp, _vp, _vp, ctypes.c_int32, _i64, _vp]),
    "birkhoff4_sinkhorn": (_int, [_vp, _vp, _int, _i64, _vp]),
    "birkhoff4_sinkhorn_bf16": (_int, [_vp, _vp, _int, _i64, _vp]),
    "birkhoff4_strerror": (ctypes.c_char_p, [_int]),
    "birkhoff4_version": (_int, []),
    "birkhoff4_last_cuda_error": (_int, []),
    "birkhoff4_device_status": (_int, [ctypes.POINTER(ctypes.c_uint), _int]),
    "birkhoff4_selftest_wait_timeout": (_int, [_i64]),
    "birkhoff4_mufu_probe": (_int, [ctypes.POINTER(ctypes.c_float), _int, _int, _vp]),
}

# The functions of hc_block.h and adamw.h.
BLOCK_SIGNATURES = {
    "hcb_workspace_bytes": (ctypes.c_size_t, [_i64, ctypes.c_int32, ctypes.c_int32]),
    "hcb_enter": (_int, [_vp, _vp]),
    "hcb_enter_backward": (_int, [_vp, _vp]),
    "hcb_leave": (_int, [_vp, _vp]),
    "hcb_leave_backward": (_int, [_vp, _vp]),
    "adamw_step": (_int, [_vp, ctypes.c_int32, _vp, _vp]),
}

HCB_MAX_STREAMS, HCB_MAX_CHANNELS = 8, 16384
HCB_ACT_NONE, HCB_ACT_SIGMOID, HCB_ACT_SILU, HCB_ACT_LINEAR = 0, 1, 2, 3
ADAMW_BLOCK = 128


def _fields(kind, names):
    return [(n, kind) for n in names.split()]


class HcbArgs(ctypes.Structure):
    """hcb_args."""
    _fields_ = (
        _fields(_i64, "T") + _fields(ctypes.c_int32, "S C x_dtype y_dtype w_dtype wn_dtype p_dtype a_dtype b_dtype act norm")
        + _fields(ctypes.c_float, "eps eps_next scale")
        + _fields(_vp, "x y gate P a b w w_next dout dh dres out_in")
        + _fields(_i64, "x_ts x_ss y_ts gate_ts P_ts a_ts b_ts dout_ts dout_ss dh_ts dres_ts dres_ss out_ts out_ss")
        + _fields(_vp, "h out dx dy dgate dP da db dw dw_next workspace")
        + _fields(ctypes.c_size_t, "workspace_bytes"))


class AdamwTensor(ctypes.Structure):
    """adamw_tensor."""
    _fields_ = _fields(_vp, "p g m v m_scale v_scale master") + _fields(_i64, "n")


class AdamwOpts(ctypes.Structure):
    """adamw_opts."""
    _fields_ = (_fields(ctypes.c_int32, "p_dtype g_dtype state_bits") + _fields(ctypes.c_double, "lr beta1 beta2 eps weight_decay")
                + _fields(_i64, "step") + _fields(_vp, "grad_scale"))


class Opts(ctypes.Structure):
    """birkhoff4_opts."""
    _fields_ = [
        ("in_dtype", ctypes.c_int32),
        ("out_dtype", ctypes.c_int32),
        ("max_evals", ctypes.c_int32),
        ("tol", ctypes.c_float),
        ("evals_out", ctypes.c_void_p),
        ("nonconv_count", ctypes.c_void_p),
        ("schedule", ctypes.c_int32),
    ]


class Birkhoff4Error(RuntimeError):
    pass


def lib():
    """The loaded library (built with nvcc on first use if missing or stale)."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        path = _build.build()
        if not os.path.exists(path):
            raise Birkhoff4Error("libbirkhoff4.so was not built")
        handle = ctypes.CDLL(path)
        for name, (res, args) in {**SIGNATURES, **BLOCK_SIGNATURES}.items():
            fn = getattr(handle, name)
            fn.restype = res
            fn.argtypes = args
        _lib = handle
        return handle


_binding = None


class _NoBinding:
    """Stands in for the extension module: no call is one that it takes."""

    def __getattr__(self, name):
        return lambda *args: None


def _load_binding(handle):
    loader = importlib.machinery.ExtensionFileLoader("_block_binding", _build.build_binding())
    spec = importlib.util.spec_from_loader("_block_binding", loader)
    module = importlib.util.module_from_spec(spec)
    loader.exec_module(module)
    module.init(*[ctypes.cast(getattr(handle, name), ctypes.c_void_p).value for name in (
        "hcb_enter", "hcb_enter_backward", "hcb_leave", "hcb_leave_backward", "hcb_workspace_bytes")])
    return module


def binding():
    """The extension module that makes the plain calls of the block and
    optimizer entry points (built and loaded on first use); where it cannot be
    built or loaded, a stand-in that leaves every call to the Python code."""
    global _binding
    if _binding is None:
        handle = lib()
        try:
            _binding = _load_binding(handle)
        except (RuntimeError, ImportError) as e:
            _build.without_binding(e)
            _binding = _NoBinding()
    return _binding


def library_path() -> str:
    return _build.LIB_PATH


def check(status: int, what: str) -> None:
    if status != B4_OK:
        L = lib()
        msg = L.birkhoff4_strerror(status).decode()
        if status == B4_ECUDA:
            msg += " (cudaError %d)" % L.birkhoff4_last_cuda_error()
        raise Birkhoff4Error("%s: %s" % (what, msg))
