"""Builds libxattn.so in-tree (bwd_xattn_fwd_gb300/_build/) with nvcc for sm_103a.

Each .cu file compiles in parallel to an object; the objects link into one shared
library with the CUDA runtime linked statically (so the library loads on a machine
without a GPU driver; the driver is reached at the first CUDA call).

csrc/xattn_torch.cpp, the native part of the binding's tensor-level calls, compiles beside them
against the installed torch and the running Python (its file carries both versions: another torch
or Python builds another; without a torch for CUDA there is none).

`--debug` (build(debug=True)) builds the same library with XATTN_DEBUG -- on-device bounds
checks that report XATTN_ERR_DEVICE_BOUNDS -- into _build_debug/ (load it by pointing
XATTN_LIBRARY at it).
"""
from __future__ import annotations

import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libxattn.so")
BUILD_DEBUG = os.path.join(HERE, "_build_debug")
LIB_DEBUG = os.path.join(BUILD_DEBUG, "libxattn.so")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
          f"-I{INCLUDE}"]


def nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found (needed to build libxattn)")
    return cand


TORCH_SRC = os.path.join(CSRC, "xattn_torch.cpp")


def torch_dir():
    """Where torch is installed (found without importing it), or None."""
    spec = importlib.util.find_spec("torch")
    return spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None


def torch_lib() -> str:
    """The native part of the tensor-level calls for the installed torch and this Python's ABI
    ("" without a torch for CUDA)."""
    if not torch_dir() or not os.path.exists(os.path.join(torch_dir(), "lib", "libc10_cuda.so")):
        return ""
    version = f"{importlib.metadata.version('torch')}.{sysconfig.get_config_var('SOABI')}"
    return os.path.join(BUILD, f"xattn_torch-{version}.so")


def _torch_current() -> bool:
    lib = torch_lib()
    if not lib:
        return True
    deps = (TORCH_SRC, os.path.join(INCLUDE, "xattn.h"))
    return os.path.exists(lib) and all(os.path.getmtime(d) <= os.path.getmtime(lib) for d in deps)


def _torch_command(out: str):
    t = torch_dir()
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    return [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", f"-I{INCLUDE}",
            f"-I{os.path.join(t, 'include')}", f"-I{os.path.join(t, 'include', 'torch', 'csrc', 'api', 'include')}",
            f"-I{os.path.join(cuda, 'include')}", f"-I{sysconfig.get_paths()['include']}", TORCH_SRC, "-o", out,
            f"-L{os.path.join(t, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    return sources() + [os.path.join(CSRC, f) for f in os.listdir(CSRC)
                        if f.endswith((".cuh", ".h"))] + [os.path.join(INCLUDE, "xattn.h")]


def up_to_date(lib: str = LIB) -> bool:
    if not os.path.exists(lib):
        return False
    t = os.path.getmtime(lib)
    return all(os.path.getmtime(d) <= t for d in _deps())


def build(force: bool = False, verbose: bool = False, extra=(), debug: bool = False) -> str:
    build_dir, lib = (BUILD_DEBUG, LIB_DEBUG) if debug else (BUILD, LIB)
    if debug:
        extra = (*extra, "-DXATTN_DEBUG")
    torch_tmp = ""
    procs = []
    if torch_lib() and (force or not _torch_current()):
        os.makedirs(BUILD, exist_ok=True)
        torch_tmp = torch_lib() + f".tmp{os.getpid()}"
        procs.append((TORCH_SRC, subprocess.Popen(_torch_command(torch_tmp), stdout=subprocess.PIPE,
                                                  stderr=subprocess.STDOUT)))
    current = not force and up_to_date(lib)
    if current and not procs:
        return lib
    os.makedirs(build_dir, exist_ok=True)
    nv = nvcc()
    objs = []
    for src in [] if current else sources():
        obj = os.path.join(build_dir, os.path.basename(src)[:-3] + ".o")
        cmd = [nv, *ARCH, *CFLAGS, *extra, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
        objs.append(obj)
    failed = []
    for src, p in procs:
        out, _ = p.communicate()
        text = out.decode(errors="replace")
        if p.returncode != 0:
            failed.append((src, text))
        elif verbose and text.strip():
            print(text, flush=True)
    if failed:
        msg = "\n".join(f"--- {s}\n{t}" for s, t in failed)
        raise RuntimeError(f"the compiler failed:\n{msg}")
    if torch_tmp:
        os.replace(torch_tmp, torch_lib())
    if current:
        return lib
    tmp = lib + f".tmp{os.getpid()}"
    cmd = [nv, *ARCH, "-shared", "--cudart", "static", "-o", tmp, *objs]
    if verbose:
        print(" ".join(cmd), flush=True)
    subprocess.run(cmd, check=True)
    os.replace(tmp, lib)
    return lib


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else [], debug="--debug" in sys.argv))
