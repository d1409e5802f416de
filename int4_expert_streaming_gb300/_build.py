"""Build libmoe.so in-tree with nvcc for sm_103a (no torch extension machinery).

Each translation unit compiles in parallel into _build/, then one nvcc link
produces int4_expert_streaming_gb300/libmoe.so (static CUDA runtime).  gcc
builds _call.so beside it, the Python module that marshals the arguments of
the operators without a context (csrc/binding.c, linked against libmoe.so, and
csrc/tensor.cc, which reads torch's tensors and is compiled with its headers).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
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
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmoe.so")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")) + glob.glob(os.path.join(CSRC, "*.cpp")))


def _torch() -> str:
    spec = importlib.util.find_spec("torch")  # without importing it
    if spec is None or not spec.origin:
        raise RuntimeError("torch not found: its headers are required to build _call.so")
    return os.path.dirname(spec.origin)


def _deps():
    return sources() + [BINDING, TENSOR, os.path.join(_torch(), "version.py")] + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + [os.path.join(ROOT, "include", "moe.h"),
                                                               os.path.abspath(__file__)]


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALL):
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALL))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD, exist_ok=True)
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

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 4)) as ex:
        tensor = ex.submit(_compile_tensor)
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
    _build_binding(tensor.result())
    return LIB


def _compile_tensor() -> str:
    obj = os.path.join(BUILD, "tensor.cc.o")
    inc = os.path.join(_torch(), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-c", TENSOR, "-o", obj, "-I" + sysconfig.get_paths()["include"], "-isystem", inc,
           "-isystem", os.path.join(inc, "torch", "csrc", "api", "include")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on tensor.cc:\n{r.stdout}\n{r.stderr}")
    return obj


def _build_binding(tensor: str) -> None:
    tmp = CALL + f".tmp{os.getpid()}"
    cmd = ["gcc", "-O2", "-Wall", "-shared", "-fPIC", "-I" + sysconfig.get_paths()["include"],
           "-I" + os.path.join(ROOT, "include"), BINDING, tensor, "-o", tmp, "-L" + PKG, "-l:" + os.path.basename(LIB),
           "-L" + os.path.join(_torch(), "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lstdc++",
           "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + os.path.join(_torch(), "lib")]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"gcc failed on binding.c:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALL)


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
