"""Build step of the CUDA library ``libmt.so`` (sm_103a), in-tree.

Each ``csrc/*.cu`` file is compiled by nvcc in parallel for
``-gencode arch=compute_103a,code=sm_103a`` and linked into
``update_merged_table_gb300/_build/libmt.so`` with the CUDA runtime linked
statically, so the library depends on nothing but the driver.

Beside it, ``csrc/py/mt_block_py.cpp`` becomes ``_build/_mt_block.so``, the
Python module through which ``block.py`` calls the library (it needs torch's
and Python's headers; without torch only the library is built).
"""
from __future__ import annotations

import glob
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(BUILD, "libmt.so")
BINDING_SRC = os.path.join(CSRC, "py", "mt_block_py.cpp")
BINDING = os.path.join(BUILD, "_mt_block.so")
BINDING_FOR = os.path.join(BUILD, "_mt_block.for")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2", "-I", INCLUDE, "-I", CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA library cannot be built")


def _newest(paths) -> float:
    return max(os.path.getmtime(p) for p in paths)


def _made_for(torch_dir: str) -> str:
    """What a Python module was compiled against: it fits this torch and this Python only."""
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "?"
    return f"torch {version} in {torch_dir}\nPython {sys.version}\n"


def _start_binding(force: bool, verbose: bool):
    """Start compiling the Python module if it is out of date; (process, file to rename, what it is made for), or None
    where there is nothing to do or no torch to make it for."""
    spec = importlib.util.find_spec("torch")
    if spec is None or spec.origin is None:
        return None
    torch_dir = os.path.dirname(spec.origin)
    made_for = _made_for(torch_dir)
    deps = [BINDING_SRC, os.path.join(INCLUDE, "mt.h"), __file__]
    if not force and os.path.exists(BINDING) and os.path.exists(BINDING_FOR) and os.path.getmtime(BINDING) >= _newest(deps):
        with open(BINDING_FOR) as f:
            if f.read() == made_for:
                return None
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    lib = os.path.join(torch_dir, "lib")
    tmp = BINDING + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", BINDING_SRC, "-o", tmp, "-I", INCLUDE,
           "-I", os.path.join(torch_dir, "include"), "-I", os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-I", sysconfig.get_paths()["include"],
           "-L", lib, f"-Wl,-rpath,{lib}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    if verbose:
        print(" ".join(cmd))
    return subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT), tmp, made_for


def _finish_binding(started):
    if started is None:
        return
    proc, tmp, made_for = started
    out, _ = proc.communicate()
    if proc.returncode != 0:
        raise RuntimeError("the Python module failed to compile:\n" + out.decode(errors="replace"))
    os.replace(tmp, BINDING)
    with open(BINDING_FOR, "w") as f:
        f.write(made_for)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link libmt.so and the Python module if any source or header is newer; return libmt.so's path."""
    os.makedirs(BUILD, exist_ok=True)
    binding = _start_binding(force, verbose)
    try:
        return _build_lib(force, verbose)
    finally:
        _finish_binding(binding)


def _build_lib(force: bool, verbose: bool) -> str:
    sources = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    headers = sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h")))
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _newest(sources + headers + [__file__]):
        return LIB
    cc = nvcc()
    procs = []
    objs = []
    for src in sources:
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        cmd = [cc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
        if verbose:
            print(" ".join(cmd))
        procs.append((src, subprocess.Popen(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT)))
    failed = []
    for src, pr in procs:
        out, _ = pr.communicate()
        if pr.returncode != 0:
            failed.append(f"{src}:\n{out.decode(errors='replace')}")
    if failed:
        raise RuntimeError("nvcc failed:\n" + "\n".join(failed))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs, "-lrt", "-lpthread", "-ldl"]
    subprocess.check_call(cmd)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
