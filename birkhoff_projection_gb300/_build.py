"""Build libbirkhoff4.so in-tree with nvcc for sm_103a (GB300).

The kernel translation units compile in parallel; the shared library links
the CUDA runtime statically, so it needs nothing from PyTorch at load time.
Beside it, g++ builds a small extension module against PyTorch's headers, the
short way from Python into the library's block and optimizer entry points.
The library does not need it, and neither do the operators: without it their
calls take longer.  It is of one Python and one PyTorch, which its name says.

    python -m birkhoff_projection_gb300._build [--force] [-v]
"""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libbirkhoff4.so")
BINDING_SOURCE = os.path.join(CSRC, "block_binding.cpp")

SOURCES = ["birkhoff4_api.cu", "k_forward.cu", "k_backward.cu", "k_fused.cu", "k_sinkhorn.cu",
           "birkhoff4_noalloc.cu", "k_nxn.cu", "eot_stream.cu",
           "eot_transport.cu", "k_mapped.cu", "hcb_api.cu", "hcb_enter.cu", "hcb_leave.cu",
           "hcb_leave_bwd.cu", "hcb_leave_enter_bwd.cu", "hcb_residual.cu", "adamw.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
              "-I", CSRC, "-I", INCLUDE]


def nvcc() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def binding_path() -> str:
    """Where the extension module for the running Python and PyTorch is."""
    import torch

    return os.path.join(PKG, "_block_binding.%s.torch-%s.so" % (sysconfig.get_config_var("SOABI"), torch.__version__))


def _up_to_date(path, inputs) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in inputs)


def _headers():
    return [os.path.join(INCLUDE, h) for h in os.listdir(INCLUDE)] + [os.path.abspath(__file__)]


def library_up_to_date() -> bool:
    return _up_to_date(LIB_PATH, [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")] + _headers())


def binding_up_to_date() -> bool:
    return _up_to_date(binding_path(), [BINDING_SOURCE] + _headers())


def _run(cmd, what: str, verbose: bool = False) -> None:
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError("%s failed: %s" % (what, e)) from e
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))
    if verbose:
        sys.stderr.write(r.stdout + r.stderr)


def build_binding(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of the extension module."""
    path = binding_path()
    if not force and binding_up_to_date():
        return path
    import torch

    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    include = [INCLUDE, os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    tmp = path + ".tmp%d" % os.getpid()
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI]
         + ["-I" + d for d in include] + [BINDING_SOURCE, "-o", tmp, "-L" + lib, "-Wl,-rpath," + lib,
                                          "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch", "-ltorch_python"],
         "g++ of block_binding.cpp", verbose)
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if stale) and return the path of libbirkhoff4.so."""
    if not force and library_up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose else []
    # tile-shape and pipeline macros for measurement sweeps, e.g.
    # B4_NVCC_DEFINES="B4_FWD_TILE=256 B4_FWD_NSTAGE=3"
    extra += ["-D" + d for d in os.environ.get("B4_NVCC_DEFINES", "").split()]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        _run([nvcc()] + ARCH + NVCC_FLAGS + extra + ["-c", os.path.join(CSRC, src), "-o", obj], "nvcc of " + src, verbose)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    _run([nvcc()] + ARCH + ["-shared", "-o", tmp] + objs, "nvcc link")
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


def without_binding(why) -> None:
    warnings.warn("no _block_binding: the block operators' and the optimizer's calls go through Python code, which takes "
                  "longer (%s)" % why, RuntimeWarning, stacklevel=3)


def build_all(force: bool = False, verbose: bool = False) -> str:
    """build and build_binding side by side; the library's path.  Without the
    extension module: a warning."""
    with ThreadPoolExecutor(max_workers=1) as ex:
        binding = ex.submit(build_binding, force, verbose)
        path = build(force, verbose)
        try:
            binding.result()
        except RuntimeError as e:
            without_binding(e)
    return path


if __name__ == "__main__":
    build_all(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB_PATH)
