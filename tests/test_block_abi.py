"""The C ABI of hc_block.h and adamw.h, and their Python bindings' checks, on
the host: symbols, struct layouts, and every refusal (nothing is launched, so
these run without a GPU)."""
import ctypes
import os
import re

import pytest
import torch

from birkhoff_projection_gb300 import _lib, block, optim
from birkhoff_projection_gb300._lib import B4_BF16, B4_EINVAL, B4_ENOTIMPL, B4_F32, B4_OK

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
FAKE = 0x10000  # never dereferenced: refused before use


@pytest.fixture(scope="module")
def L():
    return _lib.lib()


def header(name):
    return re.sub(r"/\*.*?\*/", "", open(os.path.join(ROOT, "include", name)).read(), flags=re.S)


def test_every_declared_function_is_bound(L):
    names = set()
    for h in ("hc_block.h", "adamw.h"):
        names |= set(re.findall(r"\b((?:hcb|adamw)_\w+)\s*\(", header(h)))
    assert names == set(_lib.BLOCK_SIGNATURES)
    for n in names:
        assert hasattr(L, n)


@pytest.mark.parametrize("struct,name,cls", [("hc_block.h", "hcb_args", _lib.HcbArgs),
                                             ("adamw.h", "adamw_tensor", _lib.AdamwTensor),
                                             ("adamw.h", "adamw_opts", _lib.AdamwOpts)])
def test_structures_have_the_headers_fields_in_order(struct, name, cls):
    body = re.search(r"typedef struct \{([^}]*)\} %s;" % name, header(struct)).group(1)
    kinds = {"int64_t": ctypes.c_int64, "int32_t": ctypes.c_int32, "float": ctypes.c_float, "double": ctypes.c_double,
             "size_t": ctypes.c_size_t}
    fields = []
    for line in body.split(";"):
        line = line.strip()
        if line:
            kind, names = re.match(r"((?:const )?\w+) (.*)", line, flags=re.S).groups()
            for n in names.split(","):
                n = n.strip()
                fields.append((n.lstrip("*"), ctypes.c_void_p if n.startswith("*") else kinds[kind]))
    assert fields == list(cls._fields_)


def test_packed_arguments_have_the_structures_layout():
    kinds = {ctypes.c_int64: "q", ctypes.c_int32: "i", ctypes.c_float: "f", ctypes.c_void_p: "Q", ctypes.c_size_t: "Q"}
    flat = re.sub(r"(\d+)(\w)", lambda m: m.group(2) * int(m.group(1)), block._ARGS.format[1:])
    assert flat == "".join("Q" if k is ctypes.c_size_t or k is ctypes.c_void_p else kinds[k] for _, k in _lib.HcbArgs._fields_)
    assert block._ARGS.size == ctypes.sizeof(_lib.HcbArgs)
    numbers = list(range(1, len(flat) + 1))
    args = _lib.HcbArgs.from_buffer_copy(block._ARGS.pack(*numbers))
    assert [getattr(args, n) for n, _ in _lib.HcbArgs._fields_] == numbers


def test_packed_optimizer_arguments_have_the_structures_layout():
    assert ctypes.sizeof(_lib.AdamwTensor) == 8 * optim._FIELDS
    o = _lib.AdamwOpts.from_buffer_copy(optim._OPTS.pack(*range(1, 11)))
    assert [getattr(o, n) for n, _ in _lib.AdamwOpts._fields_] == list(range(1, 11))


def test_constants_match():
    text = open(os.path.join(ROOT, "include", "hc_block.h")).read() + open(os.path.join(ROOT, "include", "adamw.h")).read()
    for name in ("HCB_MAX_STREAMS", "HCB_MAX_CHANNELS", "HCB_ACT_NONE", "HCB_ACT_SIGMOID", "HCB_ACT_SILU",
                 "HCB_ACT_LINEAR", "ADAMW_BLOCK"):
        assert int(re.search(r"#define %s (\d+)" % name, text).group(1)) == getattr(_lib, name)


ENTRIES = {
    "hcb_enter": dict(x=FAKE, h=FAKE),
    "hcb_enter_backward": dict(x=FAKE, dh=FAKE, dx=FAKE),
    "hcb_leave": dict(x=FAKE, y=FAKE, out=FAKE),
    "hcb_leave_backward": dict(dout=FAKE, x=FAKE, y=FAKE, dx=FAKE, dy=FAKE),
}


def call(L, name, **kw):
    a = _lib.HcbArgs(T=4, S=4, C=64, norm=1)
    for k, v in (ENTRIES[name] | kw).items():
        setattr(a, k, v)
    return getattr(L, name)(ctypes.byref(a), None)


@pytest.mark.parametrize("name", sorted(ENTRIES))
def test_block_entries_refuse_bad_sizes_and_types(L, name):
    bad = [dict(T=-1), dict(T=2**31), dict(x_ts=2**29), dict(b_ts=2**40), dict(S=0), dict(S=9), dict(C=0), dict(C=16385), dict(x_dtype=2), dict(y_dtype=-1),
           dict(w_dtype=5), dict(wn_dtype=2), dict(p_dtype=2), dict(a_dtype=2), dict(b_dtype=2), dict(eps=-1.0),
           dict(eps=float("nan")), dict(eps=float("inf")), dict(eps_next=-1.0), dict(scale=float("inf")),
           dict(scale=float("nan")), dict(act=4), dict(act=-1), dict(x_ts=-1), dict(x_ss=-4), dict(y_ts=-1),
           dict(gate_ts=-1), dict(P_ts=-1), dict(a_ts=-1), dict(b_ts=-1), dict(dout_ts=-1), dict(dout_ss=-1),
           dict(dh_ts=-1), dict(dres_ts=-1), dict(dres_ss=-1), dict(out_ts=-1), dict(out_ss=-1)]
    for kw in bad:
        assert call(L, name, **kw) == B4_EINVAL, kw
    assert call(L, name, x_dtype=B4_BF16, y_dtype=B4_F32) == B4_ENOTIMPL
    assert getattr(L, name)(None, None) == B4_EINVAL


@pytest.mark.parametrize("name", sorted(ENTRIES))
def test_block_entries_refuse_missing_and_misplaced_pointers(L, name):
    for k in ENTRIES[name]:
        if name == "hcb_enter_backward" and k == "dx" or name == "hcb_leave_backward" and k in ("x", "dx", "dy"):
            continue  # optional there
        assert call(L, name, **{k: None}) == B4_EINVAL, k
        assert call(L, name, **{k: FAKE + 2}) == B4_EINVAL, k  # fp32 at half its size
    for k in ("P", "a", "b", "w", "w_next", "dP", "da", "db", "dw", "dw_next"):
        assert call(L, name, **{k: FAKE + 2}) == B4_EINVAL, k
    assert call(L, name, T=0, **{k: None for k in ENTRIES[name]}) == B4_OK


def test_block_entries_refuse_gradients_of_what_is_not_there(L):
    assert call(L, "hcb_enter_backward", da=FAKE) == B4_EINVAL
    assert call(L, "hcb_enter_backward", dx=None, dres=FAKE) == B4_EINVAL
    for kw in (dict(P=FAKE, x=None), dict(dP=FAKE), dict(db=FAKE), dict(dgate=FAKE), dict(dh=FAKE),
               dict(dh=FAKE, out_in=FAKE, dx=None), dict(dh=FAKE, out_in=FAKE, da=FAKE)):
        assert call(L, "hcb_leave_backward", **kw) == B4_EINVAL, kw
    for name in ("hcb_leave", "hcb_leave_backward"):
        assert call(L, name, gate=FAKE) == B4_EINVAL  # a gate needs its act
        assert call(L, name, act=1) == B4_EINVAL  # and an act its gate


def test_block_workspace(L):
    assert L.hcb_workspace_bytes(0, 64, 1) == 0
    assert L.hcb_workspace_bytes(4, 64, 0) == 0
    assert L.hcb_workspace_bytes(4, 64, 3) == 0
    assert L.hcb_workspace_bytes(4, 16385, 1) == 0
    one = L.hcb_workspace_bytes(4, 64, 1)
    assert one >= 4 * 64 and L.hcb_workspace_bytes(4, 64, 2) == 2 * one
    for name in ("hcb_enter_backward", "hcb_leave_backward"):
        assert call(L, name, dw=FAKE) == B4_EINVAL
        assert call(L, name, dw=FAKE, workspace=FAKE, workspace_bytes=one - 1) == B4_EINVAL
        assert call(L, name, dw=FAKE, workspace=FAKE + 4, workspace_bytes=one) == B4_EINVAL


def step(L, tensors=None, count=1, **kw):
    t = (_lib.AdamwTensor * 2)(_lib.AdamwTensor(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 256),
                               _lib.AdamwTensor(FAKE, FAKE, FAKE, FAKE, FAKE, FAKE, None, 256))
    for k, v in (tensors or {}).items():
        setattr(t[count - 1], k, v)
    o = _lib.AdamwOpts(p_dtype=B4_F32, g_dtype=B4_F32, state_bits=8, lr=1e-3, beta1=0.9, beta2=0.99, eps=1e-8,
                       weight_decay=0.1, step=1)
    for k, v in kw.items():
        setattr(o, k, v)
    return L.adamw_step(t, count, ctypes.byref(o), None)


def test_adamw_refusals(L):
    nan, inf = float("nan"), float("inf")
    for kw in (dict(p_dtype=2), dict(g_dtype=-1), dict(state_bits=16), dict(beta1=1.0), dict(beta1=-0.1),
               dict(beta2=1.0), dict(beta2=nan), dict(lr=-1.0), dict(lr=inf), dict(lr=nan), dict(eps=-1e-9),
               dict(weight_decay=-1.0), dict(weight_decay=inf), dict(step=0), dict(grad_scale=FAKE + 1)):
        assert step(L, **kw) == B4_EINVAL, kw
    for k in ("p", "g", "m", "v", "m_scale", "v_scale"):
        for count in (1, 2):  # nothing is launched for the first tensor either
            assert step(L, {k: None}, count) == B4_EINVAL, k
    for k in ("p", "g", "m_scale", "v_scale", "master"):
        assert step(L, {k: FAKE + 2}) == B4_EINVAL, k
    assert step(L, {"m": FAKE + 2}, state_bits=32) == B4_EINVAL
    assert step(L, {"v": FAKE + 1}, state_bits=32) == B4_EINVAL
    assert step(L, {"n": -1}) == B4_EINVAL
    assert step(L, {"master": FAKE}, 2, p_dtype=B4_BF16) == B4_EINVAL  # all or none
    assert step(L, {"master": FAKE}) == B4_ENOTIMPL
    assert L.adamw_step(None, 1, ctypes.byref(_lib.AdamwOpts()), None) == B4_EINVAL
    assert L.adamw_step(None, 0, None, None) == B4_EINVAL
    assert step(L, count=-1) == B4_EINVAL
    assert step(L, {"n": 0, "p": None}) == B4_OK  # no elements: nothing to do


def test_the_short_way_takes_nothing_that_is_not_plain():
    m = _lib.binding()
    x = torch.zeros(3, 4, 8)
    y = torch.zeros(3, 8)
    for bad in (x, None, 1, "x", [x]):
        assert m.enter(bad, None, None, 1e-6, -1) is None
        assert m.enter_backward(y, bad, None, None, 1e-6, None) is None
        assert m.leave(bad, y, None, None, None, 1, None, True, 1.0, 1e-6, False, None, None, 0.0) is None
        assert m.leave_backward(bad, y, None, None, None, 1, None, True, 1.0, 1e-6, x, None, None, None, None, 0.0) is None
    assert m.adamw_table([x], b"", 0, 0) is None and m.adamw_table([], b"", 0, 0) is None
    assert m.adamw_table([x], bytes(64), 0, 0) is None and m.adamw_table((x,), bytes(64), 0, 0) is None
    for f in (m.enter, m.enter_backward, m.leave, m.leave_backward, m.adamw_table, m.init):
        with pytest.raises(TypeError):
            f(x)


def test_python_refuses_tensors_off_the_gpu():
    x, y = torch.zeros(3, 4, 8), torch.zeros(3, 8)
    for f in (lambda: block.enter(x), lambda: block.leave(x, y), lambda: block.leave_enter(x, y),
              lambda: block.enter_backward(y, x), lambda: block.leave_backward(x, x, y),
              lambda: block.leave_enter_backward(x, y, x, x, y)):
        with pytest.raises(ValueError, match="CUDA"):
            f()
    with pytest.raises(TypeError):
        block.enter([1.0])
    with pytest.raises(TypeError):
        block.enter(x.half())
    with pytest.raises(ValueError, match="CUDA"):
        optim.AdamW([torch.nn.Parameter(x)])


def test_python_refuses_bad_hyperparameters():
    p = [torch.nn.Parameter(torch.zeros(4))]
    for kw in (dict(lr=-1.0), dict(lr=float("nan")), dict(eps=-1.0), dict(weight_decay=float("inf")),
               dict(betas=(1.0, 0.9)), dict(betas=(0.9,)), dict(state_bits=16)):
        with pytest.raises(ValueError):
            optim.AdamW(p, **kw)
