"""Build libmoe.so in-tree with nvcc for sm_103a (no torch extension machinery).

Each translation unit compiles in parallel into _build/, then one nvcc link
produces int4_expert_streaming_gb300/libmoe.so (static CUDA runtime).  gcc
builds _call.so beside it, the Python module that marshals the arguments of
the operators without a context (csrc/binding.c, linked against libmoe.so, and
csrc/tensor.cc, which reads torch's tensors and is compiled with its headers).
Where torch is not installed that module is left out; libmoe.so needs none.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import re
import shutil
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
CALL = os.path.join(PKG, "_call.so")
BINDING = os.path.join(CSRC, "binding.c")
TENSOR = os.path.join(CSRC, "tensor.cc")
STAMP = os.path.join(BUILD, "binding.txt")  # what _call.so was built for
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _torch() -> str | None:
    """torch's folder, found without importing it; None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    return os.path.dirname(spec.origin) if spec and spec.origin else None


def built_for(torch_version: str) -> str:
    """What _call.so is tied to: it reads torch's tensors and Python's objects where these versions have their parts."""
    return f"torch {torch_version}, {sysconfig.get_config_var('SOABI')}"


def _built_for(torch: str) -> str:
    with open(os.path.join(torch, "version.py")) as f:
        version = re.search(r"^__version__ = ['\"](.*)['\"]", f.read(), re.M)
    if version is None:
        raise RuntimeError(f"{f.name} does not say torch's version")
    return built_for(version[1])


def _stamp(torch: str) -> str:
    return f"{_built_for(torch)}, {torch}\n"  # and where it looks for torch's libraries


def _current(made, *deps) -> bool:
    deps += (os.path.join(ROOT, "include", "moe.h"), os.path.abspath(__file__))
    return os.path.exists(made) and all(os.path.getmtime(p) <= os.path.getmtime(made) for p in deps)


def _lib_current() -> bool:
    return _current(LIB, *sources(), *glob.glob(os.path.join(CSRC, "*.h")), *glob.glob(os.path.join(CSRC, "*.cuh")))


def _binding_current(torch: str) -> bool:
    if not os.path.exists(STAMP) or not _current(CALL, BINDING, TENSOR, os.path.join(CSRC, "tensor.h")):
        return False
    with open(STAMP) as f:
        return f.read() == _stamp(torch)


def up_to_date() -> bool:
    torch = _torch()
    return _lib_current() and (torch is None or _binding_current(torch))


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    torch = _torch()
    lib, binding = force or not _lib_current(), torch is not None and (force or not _binding_current(torch))
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        tensor = ex.submit(_compile_tensor, torch) if binding else None
        if lib:
            _build_lib(ex, verbose, extra_flags)
        if binding:
            _build_binding(tensor.result(), torch)
    return LIB


def _build_lib(ex, verbose: bool, extra_flags) -> None:
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2,-Wall",
                     "-I" + os.path.join(ROOT, "include")] + list(extra_flags)

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        cmd = [nvcc] + common + ["-c", src, "-o", obj]
        if src.endswith(".cu"):
            cmd += ["-Xptxas", "-v"] if verbose else []
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, (r.stdout + r.stderr)

    results = list(ex.map(compile_one, sources()))
    if verbose:
        for _, log in results:
            if log.strip():
                print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc] + ARCH + ["-shared", "-o", tmp] + [o for o, _ in results] + ["-cudart", "static", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


def _compile_tensor(torch: str) -> str:
    obj = os.path.join(BUILD, "tensor.cc.o")
    inc = os.path.join(torch, "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", TENSOR, "-o", obj, "-I" + sysconfig.get_paths()["include"],
           f'-DMOE_BUILT_FOR="{_built_for(torch)}"', "-isystem", inc, "-isystem", os.path.join(inc, "torch", "csrc", "api", "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on tensor.cc:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_binding(tensor: str, torch: str) -> None:
    tmp, libs = CALL + f".tmp{os.getpid()}", os.path.join(torch, "lib")
    cmd = ["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"],
           "-I" + os.path.join(ROOT, "include"), BINDING, tensor, "-o", tmp, "-L" + PKG, "-l:" + os.path.basename(LIB),
           "-L" + libs, "-ltorch_python", "-ltorch_cpu", "-lc10", "-lstdc++", "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + libs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on binding.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)
    with open(tmp, "w") as f:
        f.write(_stamp(torch))
    os.replace(tmp, STAMP)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
