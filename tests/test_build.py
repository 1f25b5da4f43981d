"""The build: the library needs nvcc alone, and the extension module beside it
belongs to one Python and one PyTorch and can be done without."""
import os
import shutil
import subprocess
import sys

import pytest
import torch

from birkhoff_projection_gb300 import _build, _lib

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def alone(tmp_path, code):
    """Run code on a copy of the package, built but for its extension module, with no compiler to be found."""
    _lib.lib()
    package = os.path.join(ROOT, "birkhoff_projection_gb300")
    shutil.copytree(package, tmp_path / "birkhoff_projection_gb300",
                    ignore=shutil.ignore_patterns("_block_binding*", "__pycache__", "*.tmp*"))
    shutil.copytree(os.path.join(ROOT, "include"), tmp_path / "include")
    (tmp_path / "bin").mkdir()
    env = {**os.environ, "PATH": str(tmp_path / "bin"), "CUDA_HOME": str(tmp_path), "PYTHONPATH": str(tmp_path),
           "PYTHONWARNINGS": "always"}
    return subprocess.run([sys.executable, "-c", code], cwd=tmp_path, env=env, capture_output=True, text=True)


def test_the_library_does_without_the_extension_module(tmp_path):
    r = alone(tmp_path, "import torch, birkhoff_projection_gb300 as b4\n"
                        "from birkhoff_projection_gb300 import _build, _lib\n"
                        "print(b4.lib().birkhoff4_strerror(0).decode(), b4.__file__)\n"
                        "assert _build.build_all() == _build.build() == _build.LIB_PATH\n")
    assert r.returncode == 0, r.stderr
    assert str(tmp_path) in r.stdout
    assert "block_binding" in r.stderr and "RuntimeWarning" in r.stderr  # build_all says what it lacks


def test_the_operators_do_without_it_too(tmp_path):
    r = alone(tmp_path, "import torch\n"
                        "from birkhoff_projection_gb300 import block, _lib\n"
                        "try: block.enter(torch.zeros(2, 4, 8))\n"
                        "except ValueError as e: print(e)\n"
                        "m = _lib.binding()\n"
                        "assert m is _lib.binding() and m.adamw_table([], b'', 0, 0) is None\n")
    assert r.returncode == 0, r.stderr
    assert "CUDA" in r.stdout and r.stderr.count("RuntimeWarning") == 1


def test_the_extension_module_is_of_one_pytorch(monkeypatch):
    _lib.binding()
    mine = _build.binding_path()
    assert _build.binding_up_to_date() and os.path.exists(mine)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert _build.binding_path() != mine and not _build.binding_up_to_date()
    assert _build.library_up_to_date()


def test_a_failed_compiler_is_reported(monkeypatch, tmp_path):
    monkeypatch.setattr(_build, "binding_path", lambda: str(tmp_path / "_block_binding.so"))
    monkeypatch.setattr(_build, "BINDING_SOURCE", str(tmp_path / "nothing.cpp"))
    with pytest.raises(RuntimeError, match="block_binding"):
        _build.build_binding()
    assert os.listdir(tmp_path) == []
