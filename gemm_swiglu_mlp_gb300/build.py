"""Builds the in-tree C-ABI library libswiglu_gb300.so for sm_103a with nvcc.

    python -m gemm_swiglu_mlp_gb300.build [--force]

One translation unit, one -gencode (compute_103a -> sm_103a), static CUDA
runtime (the library needs no libcudart/libcuda at load time; the driver is
reached through cudaGetDriverEntryPointByVersion when a call needs it). Beside
it the binding module of the paged-cache calls, host C++ against the installed
PyTorch (its version is in the file's name). It is left out, with a note, where
the headers for it are missing: the library and its C ABI do not need them.
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import threading

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libswiglu_gb300.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
BINDING_SOURCE = os.path.join(CSRC, "cache_binding.cpp")


def _torch_version() -> str:
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "none"


BINDING_PATH = os.path.join(PKG_DIR, "_cache_binding_%s.so" % "".join(
    c if c.isalnum() else "_" for c in _torch_version()))
SOURCES = [os.path.join(CSRC, "swiglu_api.cu")]
DEPS = SOURCES + [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cuh")] + [
    os.path.join(INCLUDE, "swiglu.h")]


def nvcc_path() -> str:
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def nvcc_command(out_path: str, extra=()):
    return [nvcc_path(), "-gencode", "arch=compute_103a,code=sm_103a", "-lineinfo", "-O3",
            "-std=c++17", "-Xcompiler", "-fPIC", "-shared", "-I" + INCLUDE,
            "-Xptxas", "-v", *extra, "-o", out_path, *SOURCES]


def build_fault_injection_library(out_path: str) -> str:
    """Test-only build of the same sources with SWIGLU_TEST_FAULT_INJECTION:
    adds swiglu_test_set_fault_injection() and shortens the wait limit. Never
    used by the product binding; the failure-detection test loads it."""
    proc = subprocess.run(nvcc_command(out_path, extra=("-DSWIGLU_TEST_FAULT_INJECTION",)),
                          capture_output=True, text=True)
    if proc.returncode != 0:
        sys.stderr.write(proc.stdout + proc.stderr)
        raise RuntimeError("nvcc failed building the fault-injection test library")
    return out_path


def _newer(path: str, deps) -> bool:
    if not os.path.exists(path):
        return False
    t = os.path.getmtime(path)
    return all(os.path.getmtime(d) <= t for d in deps)


def up_to_date() -> bool:
    return _newer(LIB_PATH, DEPS)


def _torch_dir() -> str:
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else ""


def _cuda_dir() -> str:
    return os.path.dirname(os.path.dirname(nvcc_path())) or "/usr/local/cuda"


def binding_needs():
    """What the binding module's build needs and does not find: names, for people."""
    inc = os.path.join(_torch_dir(), "include")
    needs = [("g++", shutil.which("g++")),
             ("Python's headers", os.path.exists(
                 os.path.join(sysconfig.get_paths()["include"], "Python.h"))),
             ("PyTorch with its headers", _torch_dir() and os.path.exists(
                 os.path.join(inc, "torch", "csrc", "autograd", "python_variable.h"))),
             ("the CUDA toolkit's headers", os.path.exists(
                 os.path.join(_cuda_dir(), "include", "cuda_runtime_api.h")))]
    return [name for name, found in needs if not found]


def binding_command(out_path: str):
    """g++ on the binding module, with the installed PyTorch's headers and libraries."""
    torch_dir, cuda = _torch_dir(), _cuda_dir()
    inc = os.path.join(torch_dir, "include")
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-I" + INCLUDE, "-I" + inc,
            "-I" + os.path.join(inc, "torch", "csrc", "api", "include"),
            "-I" + os.path.join(cuda, "include"), "-I" + sysconfig.get_paths()["include"],
            "-o", out_path, BINDING_SOURCE, "-L" + os.path.join(torch_dir, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def build_binding(force: bool = False) -> str:
    if not force and _newer(BINDING_PATH, [BINDING_SOURCE, os.path.join(INCLUDE, "swiglu.h")]):
        return BINDING_PATH
    tmp = BINDING_PATH + ".tmp%d" % os.getpid()
    proc = subprocess.run(binding_command(tmp), capture_output=True, text=True)
    if proc.returncode != 0:
        sys.stderr.write(proc.stdout + proc.stderr)
        raise RuntimeError("g++ failed building %s" % os.path.basename(BINDING_PATH))
    os.replace(tmp, BINDING_PATH)
    return BINDING_PATH


def build(force: bool = False, verbose: bool = False) -> str:
    """Both, at the same time; returns the library's path. An error in either is
    raised; headers that the binding needs and that are not there only leave it out."""
    missing = binding_needs()
    if missing:
        sys.stderr.write("%s is left out (the paged-cache calls from Python need it): no %s\n"
                         % (os.path.basename(BINDING_PATH), ", no ".join(missing)))
        return build_library(force, verbose)
    errors = []

    def binding():
        try:
            build_binding(force)
        except Exception as e:  # raised below, once the library is there
            errors.append(e)

    t = threading.Thread(target=binding)
    t.start()
    try:
        path = build_library(force, verbose)
    finally:
        t.join()
    if errors:
        raise errors[0]
    return path


def build_library(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        return LIB_PATH
    tmp = LIB_PATH + ".tmp%d" % os.getpid()
    proc = subprocess.run(nvcc_command(tmp), capture_output=True, text=True)
    log = proc.stdout + proc.stderr
    with open(os.path.join(PKG_DIR, "ptxas_info.txt"), "w") as f:
        f.write(log)
    if proc.returncode != 0:
        sys.stderr.write(log)
        raise RuntimeError("nvcc failed building %s" % LIB_NAME)
    if verbose:
        sys.stderr.write(log)
    os.replace(tmp, LIB_PATH)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
